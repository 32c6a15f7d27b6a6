"""Timed cases of what surrounds the paged KV cache in a decode step: norm and rotation of queries and keys,
the cache in 8 bits, and attention over a prefix that sequences share.

Four operators: the RMS norm of each query and key head with the position rotation in the same pass (``rope``),
storing new K/V rows as 8-bit codes with a scale for each row (``append``), attention of one new token over such
a cache (``attn``), and attention of one new token for groups of sequences whose first pages are the same
(``shared``).  ``run`` computes them in plain torch operations, or through the package where ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step's token of each sequence of a batch: launch latency counts
        dict(name="rope_token", op="rope", dtype="bf16", hq=32, hkv=8, d=128, rows=64, rot=128, pairs="half", far=32768, shape=1),
        # packed prompts, slices of a joint projection
        dict(name="rope_prompt", op="rope", dtype="bf16", hq=32, hkv=8, d=128, rows=16384, rot=128, pairs="half", far=16384, shape=2),
        # an fp32 model that rotates half of each head, neighbours as pairs, far into a long context
        dict(name="rope_partial", op="rope", dtype="f32", hq=12, hkv=4, d=64, rows=5001, rot=32, pairs="next", far=1000000, shape=3),
        # the token of a decode step for every sequence of a batch
        dict(name="append_token", op="append", dtype="bf16", fmt="i8", hkv=8, d=128, batch=64, lo=1, hi=1, past=2000, page=16, shape=4),
        # packed prompts on their way into the cache
        dict(name="append_prompt", op="append", dtype="bf16", fmt="e4m3", hkv=8, d=128, batch=16, lo=64, hi=8192, past=0, page=64, shape=5),
        # one short chat turn, one sequence: the latency of a token
        dict(name="attn_one", op="attn", dtype="bf16", fmt="i8", hq=32, hkv=8, d=128, batch=1, lo=700, hi=700, page=16, shape=6),
        # a small model with fp32 queries and pages that are no power of two
        dict(name="attn_f32", op="attn", dtype="f32", fmt="e4m3", hq=8, hkv=2, d=64, batch=4, lo=1500, hi=2048, page=20, shape=7),
        # the decode benchmark's layer at a 32K context
        dict(name="attn_32k", op="attn", dtype="bf16", fmt="i8", hq=32, hkv=8, d=128, batch=8, lo=32768, hi=32768, page=64, shape=8),
        # a ragged serving batch
        dict(name="attn_ragged", op="attn", dtype="bf16", fmt="e4m3", hq=32, hkv=8, d=128, batch=32, lo=4096, hi=65536, page=16, shape=9),
        # a few samples of one short prompt, small model
        dict(name="shared_small", op="shared", hq=8, hkv=2, d=64, groups=1, members=6, shared=600, lo=1, hi=60, page=16, shape=10),
        # a few questions, some samples of each, pages that are no power of two
        dict(name="shared_groups", op="shared", hq=32, hkv=8, d=128, groups=5, members=9, shared=6000, lo=10, hi=500, page=24, shape=11),
        # a full batch behind one long document
        dict(name="shared_long", op="shared", hq=32, hkv=8, d=128, groups=1, members=64, shared=32768, lo=16, hi=1024, page=64, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["rope", "append", "attn", "attn", "shared", "shared"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    fmt = rng.choice(["i8", "e4m3"])
    page = rng.choice([8, 16, 20, 32, 48, 64, 128, 256])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    while True:
        if op == "rope":
            rot = rng.choice([d, d, d // 2, d // 4])
            case = dict(op=op, dtype=dtype, hq=g * hkv, hkv=hkv, d=d, rows=_log(rng, 1, 32768), rot=rot,
                        pairs=rng.choice(["half", "next"]), far=_log(rng, 100, 4000000), shape=shape)
            if case["rows"] * (g + 1) * hkv * d <= 16384 * 40 * 128:
                return case
        elif op == "append":
            hi = _log(rng, 1, 8192)
            batch = _log(rng, 1, 64)
            case = dict(op=op, dtype=dtype, fmt=fmt, hkv=hkv, d=d, batch=batch, lo=max(1, hi // 16), hi=hi,
                        past=rng.choice([0, _log(rng, 16, 4096)]), page=page, shape=shape)
            if batch * hi <= 65536:
                return case
        elif op == "attn":
            hi = _log(rng, 20, 65536)
            batch = _log(rng, 1, 64)
            case = dict(op=op, dtype=dtype, fmt=fmt, hq=g * hkv, hkv=hkv, d=d, batch=batch,
                        lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, page=page, shape=shape)
            if batch * hi * hkv * d <= 16 * 32768 * 8 * 128:
                return case
        else:
            groups, members = _log(rng, 1, 16), _log(rng, 2, 64)
            case = dict(op=op, hq=g * hkv, hkv=hkv, d=d, groups=groups, members=members, shared=_log(rng, 100, 32768),
                        lo=1, hi=_log(rng, 2, 2000), page=page, shape=shape)
            if (groups * members * (case["shared"] + case["hi"]) * g * hkv * d <= 64 * 33792 * 32 * 128 and groups * members <= 256
                    and groups * case["shared"] * hkv * d <= 8 * 32768 * 8 * 128):
                return case


def _lens(case):
    """(new rows, rows in all) of each sequence; the sizes come from the case alone."""
    r = random.Random(case["shape"])
    n = [_log(r, case["lo"], case["hi"]) for _ in range(case["batch"])]
    past = case.get("past", 0)
    return n, [x + (r.randint(past // 2, past) if past else 0) for x in n]


def _groups(case):
    """(sequences of each group, pages that it shares, positions of each sequence): groups differ in size."""
    r = random.Random(case["shape"])
    size = [case["members"] if i == 0 else r.randint(1, case["members"]) for i in range(case["groups"])]
    pages = [max(1, (case["shared"] if i == 0 else r.randint(case["shared"] // 2, case["shared"])) // case["page"])
             for i in range(case["groups"])]
    lens = [pages[i] * case["page"] + _log(r, case["lo"], case["hi"]) for i in range(case["groups"]) for _ in range(size[i])]
    return size, pages, lens


def _pages(case, lens):
    """A fragmented pool: (pages, table rows as lists)."""
    p = case["page"]
    need = [-(-x // p) for x in lens]
    n_pages = sum(need) + max(1, sum(need) // 10)
    ids = list(range(n_pages))
    random.Random(case["shape"] + 1).shuffle(ids)
    rows, at = [], 0
    for x in need:
        rows.append(ids[at:at + x])
        at += x
    return n_pages, rows


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op == "rope":
        n = case["rows"] * (case["hq"] + hkv)
        return {"bytes": 2 * n * d * e + 4 * case["rows"], "flops": n * (4 * d + 3 * case["rot"])}
    if op == "append":
        n = 2 * sum(_lens(case)[0]) * hkv
        return {"bytes": n * (d * e + d + 4), "flops": 2 * n * d}
    hq = case["hq"]
    if op == "attn":
        lens = _lens(case)[1]
        return {"bytes": 2 * sum(lens) * hkv * (d + 4) + len(lens) * hq * (d * (e + 4) + 4) + 4 * sum(-(-x // case["page"]) for x in lens),
                "flops": 4 * d * hq * sum(lens)}
    size, pages, lens = _groups(case)
    once = sum(pages) * case["page"]
    alone = sum(lens) - sum(m * x for m, x in zip(size, pages)) * case["page"]
    return {"bytes": 2 * (once + alone) * hkv * d * e + len(lens) * hq * (d * (e + 4) + 4) + 4 * (once + alone) // case["page"],
            "flops": 4 * d * hq * sum(lens)}


# ------------------------------------------------------------------ inputs

class State:
    pass


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(n):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return _ints(at)


def _inv_freq(rot):
    return [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def _page_bytes(case):
    return -(-case["hkv"] * case["page"] * (case["d"] + 4) // 16) * 16


def _views(pool, case):
    """Codes [pages, heads, positions, d] and scales [pages, heads, positions] of a pool of 8-bit pages."""
    h, p, d = case["hkv"], case["page"], case["d"]
    codes = pool[:, :h * p * d].view(DTYPES[case["fmt"]]).unflatten(1, (h, p, d))
    return codes, pool[:, h * p * d:h * p * (d + 4)].view(torch.float32).unflatten(1, (h, p))


def _quantise(x, fmt):
    """Codes and scales of rows [..., d]: int8 with s = amax / 127, e4m3 with the smallest power of two s for which
    amax <= 448 s; codes are the nearest to x / s (ties to even; in 64 bits, since many quotients lie at a tie)."""
    x = x.float()
    top = x.abs().amax(-1)
    if fmt == "i8":
        s = top / torch.full_like(top, 127.0)  # (by a number, torch multiplies with the rounded 1 / 127)
        c = (x.double() / torch.where(s > 0, s, 1.0).double()[..., None]).round().clamp(-127, 127).to(torch.int8)
    else:
        m, e = torch.frexp(top)
        s = torch.where(top > 0, torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875)), 0.0)
        c = (x / torch.where(s > 0, s, 1.0)[..., None]).to(torch.float8_e4m3fn)
    return c, s


def prepare(case, seed):
    s = State()
    s.case, op, d, hkv = dict(case), case["op"], case["d"], case["hkv"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype = DTYPES[case.get("dtype", "bf16")]
    if op == "rope":
        hq, n = case["hq"], case["rows"]
        joint = _randn(g, (n, hq + 2 * hkv, d), dtype)  # a projection of the hidden states: q, k and v side by side
        joint *= 0.5 + torch.rand((n, 1, 1), generator=g, device="cuda").to(dtype) * 2
        s.q, s.k = joint[:, :hq], joint[:, hq:hq + hkv]
        s.wq, s.wk = (1.0 + 0.2 * _randn(g, (d,), torch.float32)).to(dtype), (1.0 + 0.2 * _randn(g, (d,), torch.float32)).to(dtype)
        s.pos = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s.eps = 1e-6
        s.freq = torch.tensor(_inv_freq(case["rot"]), dtype=torch.float64, device="cuda")
        if own:
            import slow_sparse_kv_gb300 as sfi
            s.lay = sfi.RotaryLayout(hq, hkv, d, dtype, s.pos, rotary_dim=case["rot"], inv_freq=_inv_freq(case["rot"]),
                                     interleaved=case["pairs"] == "next", eps=s.eps)
            s.q_out = torch.empty(n, hq, d, dtype=dtype, device="cuda")
            s.k_out = torch.empty(n, hkv, d, dtype=dtype, device="cuda")
        return s
    s.page = case["page"]
    if op == "shared":
        size, shared, lens = _groups(case)
        # the group's pages, then each sequence's own behind them
        n_pages, rows = _pages(case, [x * s.page for x in shared] + [n - x * s.page for m, x, k in zip(size, shared, range(len(size)))
                                                                    for n in lens[sum(size[:k]):sum(size[:k]) + m]])
        of = [i for i, m in enumerate(size) for _ in range(m)]
        rows = [rows[i] + rows[len(size) + b] for b, i in enumerate(of)]
    else:
        new, lens = _lens(case)
        n_pages, rows = _pages(case, lens)
    s.n_pages, s.width = n_pages, max(len(r) for r in rows) + 1
    s.table = _ints([r + [-1] * (s.width - len(r)) for r in rows])
    s.len = _ints(lens)
    u = torch.nn.functional.normalize(_randn(g, (d,), torch.float32), dim=0)
    if op == "shared":
        pool = (n_pages, hkv, s.page, d)
        s.k, s.v = _randn(g, pool, dtype), _randn(g, pool, dtype)
        s.k += (3.0 * (torch.rand(pool[:3], generator=g, device="cuda") < 0.01))[..., None].to(dtype) * u.to(dtype)
        s.q = _randn(g, (len(lens), case["hq"], d), dtype) + 2.0 * u.to(dtype)
        s.cu, s.shared = _offsets(size), _ints(shared)
        s.of = torch.tensor(of, device="cuda")
        s.most, s.long, s.short = max(size), max(shared), max(len(r) - shared[i] for r, i in zip(rows, of))
    else:
        pool = (n_pages, _page_bytes(case))
        s.k, s.v = (torch.zeros(pool, dtype=torch.uint8, device="cuda") for _ in range(2))
        if op == "append":
            total = sum(new)
            s.k_new, s.v_new = _randn(g, (total, hkv, d), dtype), _randn(g, (total, hkv, d), dtype)
            s.cu = _offsets(new)
        else:
            for x, keys in ((s.k, True), (s.v, False)):  # pages at a time, to spare memory
                codes, scale = _views(x, case)
                for i in range(0, n_pages, 4096):
                    r = _randn(g, codes[i:i + 4096].shape, torch.float32)
                    if keys:
                        r += (3.0 * (torch.rand(r.shape[:3], generator=g, device="cuda") < 0.01))[..., None] * u
                    codes[i:i + 4096], scale[i:i + 4096] = _quantise(r, case["fmt"])
            s.q = _randn(g, (case["batch"], case["hq"], d), dtype) + 2.0 * u.to(dtype)
    if own:
        import slow_sparse_kv_gb300 as sfi
        s.lay = sfi.PagedLayout(case.get("hq", hkv), hkv, d, DTYPES[case.get("fmt", "bf16")], s.page, s.n_pages, s.table, s.len)
        s.ws = sfi.paged_shared_workspace(s.lay) if op == "shared" else sfi.paged_workspace(s.lay)
        if op != "append":
            s.out = torch.empty(len(lens), case["hq"], d, device="cuda")
            s.lse = torch.empty(len(lens), case["hq"], device="cuda")
    return s


# --------------------------------------------------------------------- run

def run(s):
    return (_own if own else _plain)[s.case["op"]](s)


def _plain_rope(s):
    rot = s.case["rot"]
    angle = (s.pos.double()[:, None] * s.freq)[:, None]  # (far positions need 64 bits)
    c, sn = angle.cos().float(), angle.sin().float()
    out = []
    for x, w in ((s.q, s.wq), (s.k, s.wk)):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s.eps) * w.float()
        if s.case["pairs"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            turned = torch.cat([a * c - b * sn, a * sn + b * c], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)
        out.append(torch.cat([turned, x[..., rot:]], -1).to(s.q.dtype))
    return {"q": out[0], "k": out[1]}


def _held(s):
    """Codes (whole numbers, or the 8-bit floats that they are) and scales of both pools."""
    (kc, ks), (vc, vs) = _views(s.k, s.case), _views(s.v, s.case)
    return {"k": kc, "k_scale": ks, "v": vc, "v_scale": vs}


def _plain_append(s):
    cu = s.cu.long()
    new = cu.diff()
    t = torch.arange(s.k_new.shape[0], device="cuda")
    b = torch.bucketize(t, cu[1:], right=True)
    pos = s.len.long()[b] - new[b] + t - cu[b]
    page = s.table.long()[b, pos // s.page]
    for x, pool in ((s.k_new, s.k), (s.v_new, s.v)):
        codes, scale = _views(pool, s.case)
        c, sc = _quantise(x, s.case["fmt"])
        codes.view(torch.uint8)[page, :, pos % s.page] = c.view(torch.uint8)
        scale[page, :, pos % s.page] = sc
    return _held(s)


def _softmax(score, other=None):
    """exp(score - top) in place, the row's sum and the top, of one or two blocks of scores of the same rows."""
    top = score.amax(-1, keepdim=True)
    if other is not None:
        top = torch.maximum(top, other.amax(-1, keepdim=True))
    base = top.masked_fill(top == -math.inf, 0.0)
    total = score.sub_(base).exp_().sum(-1, keepdim=True)
    if other is not None:
        total = total + other.sub_(base).exp_().sum(-1, keepdim=True)
    return total, (base + total.log()).squeeze(-1)


def _plain_attn(s):
    hq, hkv, d = s.case["hq"], s.case["hkv"], s.case["d"]
    tab = s.table.long().clamp_min(0)
    b, w = tab.shape
    k, v = (torch.mul(c.view(torch.uint8)[tab].view(c.dtype).float(), z[tab][..., None]).transpose(1, 2).reshape(b, hkv, w * s.page, d)
            for c, z in (_views(x, s.case) for x in (s.k, s.v)))
    score = s.q.float().view(b, hkv, hq // hkv, d) @ k.transpose(2, 3)
    score.mul_(1.0 / math.sqrt(d))
    score.masked_fill_((torch.arange(w * s.page, device="cuda") >= s.len[:, None])[:, None, None], -math.inf)
    total, lse = _softmax(score)
    return {"out": ((score @ v) / total).reshape(b, hq, d), "lse": lse.reshape(b, hq)}


def _plain_shared(s):
    hq, hkv, d, p = s.case["hq"], s.case["hkv"], s.case["d"], s.page
    grp, n, most = hq // hkv, s.len.shape[0], s.most
    cu, shared, tab = s.cu.long(), s.shared.long(), s.table.long().clamp_min(0)
    mine = torch.arange(n, device="cuda") - cu[s.of]  # the place in the group
    # the groups' prefixes, read once, against all their sequences' queries (padded to the largest group)
    at = torch.arange(s.long, device="cuda")
    first = tab[cu[:-1]][:, at]
    ng = first.shape[0]
    k, v = (x[first].transpose(1, 2).reshape(ng, hkv, -1, d).float() for x in (s.k, s.v))
    q = torch.zeros(ng, most, hq, d, device="cuda")
    q[s.of, mine] = s.q.float()
    q = q.view(ng, most, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(ng, hkv, most * grp, d)
    pre = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    pre.masked_fill_((torch.arange(s.long * p, device="cuda") >= shared[:, None] * p)[:, None, None], -math.inf)
    pre = pre.view(ng, hkv, most, grp, -1).transpose(1, 2)
    # each sequence's own positions
    page = (shared[s.of][:, None] + torch.arange(s.short, device="cuda")).clamp_max(s.width - 1)
    own_tab = tab.gather(1, page)
    ko, vo = (x[own_tab].transpose(1, 2).reshape(n, hkv, -1, d).float() for x in (s.k, s.v))
    post = (s.q.float().view(n, hkv, grp, d) @ ko.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    left = s.len - shared[s.of] * p
    hidden = torch.arange(s.short * p, device="cuda") >= left[:, None]
    post.masked_fill_(hidden[:, None, None], -math.inf)
    mine_pre = pre[s.of, mine]
    total, lse = _softmax(mine_pre, post)
    pre.zero_()
    pre[s.of, mine] = mine_pre
    o = pre.transpose(1, 2).reshape(ng, hkv, most * grp, -1) @ v
    o = o.view(ng, hkv, most, grp, d).transpose(1, 2)[s.of, mine] + post @ vo
    return {"out": (o / total).reshape(n, hq, d), "lse": lse.reshape(n, hq)}


_plain = {"rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "shared": _plain_shared}


def _own_rope(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_qk_norm_rope(s.lay, s.q, s.k, s.q_out, s.k_out, s.wq, s.wk)
    return {"q": s.q_out, "k": s.k_out}


def _own_append(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_paged_append_q8(s.lay, s.k_new, s.v_new, s.k, s.v, s.cu, s.ws)
    return _held(s)


def _own_attn(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_paged_attn_q8(s.lay, s.q, s.k, s.v, s.out, s.lse, s.ws)
    return {"out": s.out, "lse": s.lse}


def _own_shared(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_paged_attn_shared(s.lay, s.cu, s.shared, s.q, s.k, s.v, s.out, s.lse, s.ws)
    return {"out": s.out, "lse": s.lse}


_own = {"rope": _own_rope, "append": _own_append, "attn": _own_attn, "shared": _own_shared}


# ------------------------------------------------------------------- exact

def _exact_rope(s):
    """Each pair as a complex number, turned by e^(i angle)."""
    rot, out = s.case["rot"], {}
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), torch.outer(s.pos.double(), s.freq))[:, None]
    for name, x, w in (("q", s.q, s.wq), ("k", s.k, s.wk)):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s.eps) * w.double()
        part = x[..., :rot]
        z = torch.complex(*part.chunk(2, -1)) if s.case["pairs"] == "half" else torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous())
        z = z * turn
        part = torch.cat([z.real, z.imag], -1) if s.case["pairs"] == "half" else torch.view_as_real(z).flatten(-2)
        out[name] = torch.cat([part, x[..., rot:]], -1)
    return out


def _exact_append(s):
    """The scales are fp32 numbers by definition; codes from quotients in 64 bits, e4m3 by its steps."""
    cu, lens = s.cu.tolist(), s.len.tolist()
    out = {}
    for name, new, pool in (("k", s.k_new, s.k), ("v", s.v_new, s.v)):
        codes, scale = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in _views(pool, s.case))
        x = new.double()
        top = x.abs().amax(-1)
        if s.case["fmt"] == "i8":
            z = (top / 127).float().double()
            c = (x / z[..., None]).round()
        else:
            z = torch.exp2(torch.ceil(torch.log2(top / 448)))
            y = x / z[..., None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
            c = (y / step).round() * step
        for b, n in enumerate(lens):
            m = cu[b + 1] - cu[b]
            pos = torch.arange(n - m, n, device="cuda")
            page = s.table[b].long()[pos // s.page]
            codes[page, :, pos % s.page] = c[cu[b]:cu[b + 1]]
            scale[page, :, pos % s.page] = z[cu[b]:cu[b + 1]]
        # (int8 codes are whole numbers, which are compared as such)
        out[name], out[name + "_scale"] = None if s.case["fmt"] == "i8" else codes, scale
    return out


def _exact_attn(s, rows):
    """One sequence and KV head at a time; rows(b, h): its keys and values in 64 bits."""
    case = s.case
    grp, out, lse = case["hq"] // case["hkv"], [], []
    for b in range(s.len.shape[0]):
        for h in range(case["hkv"]):
            k, v = rows(b, h)
            t = s.q[b, h * grp:(h + 1) * grp].double() @ k.T / case["d"] ** 0.5
            lse.append(torch.logsumexp(t, -1))
            out.append(torch.exp(t - lse[-1][:, None]) @ v)
    n = s.len.shape[0]
    return {"out": torch.cat(out).view(n, case["hq"], case["d"]), "lse": torch.cat(lse).view(n, case["hq"])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if case["op"] == "append":
        return _exact_append(s)
    lens = s.len.tolist()
    pools = [_views(x, case) for x in (s.k, s.v)] if case["op"] == "attn" else None

    def rows(b, h):
        ids = s.table[b, :-(-lens[b] // s.page)].long()
        if pools is None:
            both = [x[ids, h].double() for x in (s.k, s.v)]
        else:
            both = [c[:, h].view(torch.uint8)[ids].view(c.dtype).double() * z[ids, h].double()[..., None] for c, z in pools]
        return [x.reshape(-1, case["d"])[:lens[b]] for x in both]

    return _exact_attn(s, rows)
