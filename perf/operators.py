"""Timed cases of the prompt attention and of the paged KV cache.

Four operators: causal attention over packed prompts (``prefill``), attention of one new token over
a paged cache (``paged``), storing new K/V rows in the pages (``append``) and the page bookkeeping
with its copies (``fork``: free, fork and extend sequences; ``compact``: close the holes).  ``run``
computes them in plain torch operations, or through the package where ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a few short questions of a small model served together: launch latency counts
        dict(name="prefill_short", op="prefill", hq=8, hkv=2, d=64, batch=8, lo=1, hi=200, past=0, shape=1),
        # a batch of prompts of mixed lengths packed into one call
        dict(name="prefill_packed", op="prefill", hq=32, hkv=8, d=128, batch=16, lo=64, hi=4096, past=0, shape=2),
        # the next chunk of long prompts, whose earlier chunks are context already
        dict(name="prefill_chunk", op="prefill", hq=32, hkv=8, d=128, batch=3, lo=700, hi=1100, past=12000, shape=3),
        # one long document
        dict(name="prefill_long", op="prefill", hq=32, hkv=8, d=128, batch=1, lo=16384, hi=16384, past=0, shape=4),
        # one short chat turn, one sequence: the latency of a token
        dict(name="paged_one", op="paged", dtype="bf16", hq=32, hkv=8, d=128, batch=1, lo=700, hi=700, page=16, shape=5),
        # a small fp32 model with pages that are no power of two
        dict(name="paged_f32", op="paged", dtype="f32", hq=8, hkv=2, d=64, batch=4, lo=1500, hi=2048, page=20, shape=6),
        # the decode benchmark's layer at a 32K context
        dict(name="paged_32k", op="paged", dtype="bf16", hq=32, hkv=8, d=128, batch=8, lo=32768, hi=32768, page=64, shape=7),
        # a ragged serving batch
        dict(name="paged_ragged", op="paged", dtype="bf16", hq=32, hkv=8, d=128, batch=32, lo=4096, hi=65536, page=16, shape=8),
        # the token of a decode step for every sequence of a batch
        dict(name="append_token", op="append", dtype="bf16", hkv=8, d=128, batch=64, lo=1, hi=1, past=2000, page=16, shape=9),
        # packed prompts on their way into the cache
        dict(name="append_prompt", op="append", dtype="bf16", hkv=8, d=128, batch=16, lo=64, hi=8192, past=0, page=64, shape=10),
        # a sampling step: finished sequences leave, others are forked into their slots, all grow by a token
        dict(name="pages_fork", op="fork", dtype="bf16", hkv=8, d=128, layers=8, batch=64, lo=100, hi=2000, page=64, forks=16, shape=11),
        # a fragmented pool after many requests, compacted
        dict(name="pages_compact", op="compact", dtype="bf16", hkv=8, d=128, layers=8, batch=32, lo=100, hi=1200, page=64, spare=0.6, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pairs(case):
    return sum(q * k - q * (q - 1) // 2 for q, k in zip(*_lens(case)))


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["prefill", "prefill", "paged", "paged", "append", "fork", "compact"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    page = rng.choice([8, 16, 20, 32, 48, 64, 128, 256])
    g = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
    while True:
        batch = _log(rng, 1, 48)
        if op == "prefill":
            hi = _log(rng, 4, 16384)
            lo = max(1, hi // rng.choice([1, 2, 8, 64]))
            past = rng.choice([0, 0, _log(rng, 16, 8192)])
            case = dict(op=op, hq=g * hkv, hkv=hkv, d=d, batch=batch, lo=lo, hi=hi, past=past, shape=shape)
            # the plain form holds every (row, key) score of the padded batch
            if batch * g * hkv * hi * (hi + 2 * past) <= 16384 * 16384 * 32 and _pairs(case) * g * hkv <= 16384 * 16384 * 16:
                return case
        elif op == "paged":
            hi = _log(rng, 20, 65536)
            lo = max(1, hi // rng.choice([1, 2, 16]))
            case = dict(op=op, dtype=dtype, hq=g * hkv, hkv=hkv, d=d, batch=batch, lo=lo, hi=hi, page=page, shape=shape)
            if batch * hi * hkv * d * (2 if dtype == "bf16" else 4) <= 32 * 32768 * 8 * 128 * 2:
                return case
        elif op == "append":
            hi = _log(rng, 1, 8192)
            case = dict(op=op, dtype=dtype, hkv=hkv, d=d, batch=batch, lo=max(1, hi // 16), hi=hi,
                        past=rng.choice([0, _log(rng, 16, 4096)]), page=page, shape=shape)
            if batch * hi <= 65536:
                return case
        elif op == "fork":
            batch = max(2, batch)
            case = dict(op=op, dtype=dtype, hkv=hkv, d=d, layers=rng.choice([1, 4, 8]), batch=batch, lo=50,
                        hi=_log(rng, 60, 2000), page=page, forks=rng.randint(1, max(1, batch // 3)), shape=shape)
            return case
        else:
            case = dict(op=op, dtype=dtype, hkv=hkv, d=d, layers=rng.choice([1, 4, 8]), batch=min(batch, 32), lo=50,
                        hi=_log(rng, 60, 1200), page=page, spare=rng.choice([0.1, 0.5, 1.0]), shape=shape)
            return case


def _lens(case):
    """(new rows, rows in all) of each sequence; the sizes come from the case alone."""
    r = random.Random(case["shape"])
    n = [_log(r, case["lo"], case["hi"]) for _ in range(case["batch"])]
    past = case.get("past", 0)
    return n, [x + (r.randint(past // 2, past) if past else 0) for x in n]


def _pages(case, lens, spare=0.1):
    """A fragmented pool: (pages, table rows as lists, free pages), at random from the case's sizes."""
    p = case["page"]
    need = [-(-x // p) for x in lens]
    n_pages = sum(need) + max(1, int(spare * sum(need)))
    ids = list(range(n_pages))
    random.Random(case["shape"] + 1).shuffle(ids)
    rows, at = [], 0
    for x in need:
        rows.append(ids[at:at + x])
        at += x
    return n_pages, rows


def _fork_plan(case):
    """(sequences that finish, parents of the forks): the forks take the freed slots."""
    r = random.Random(case["shape"] + 2)
    gone = sorted(r.sample(range(case["batch"]), min(case["forks"], case["batch"] - 1)))
    stay = [b for b in range(case["batch"]) if b not in gone]
    return gone, [r.choice(stay) for _ in gone]


def work(case):
    op, d, hkv = case["op"], case["d"], case["hkv"]
    new, lens = _lens(case)
    e = 4 if case.get("dtype") == "f32" else 2
    if op == "prefill":
        hq = case["hq"]
        return {"bytes": 2 * d * (2 * sum(new) * hq + 2 * sum(lens) * hkv) + 4 * sum(new) * hq, "flops": 4 * d * hq * _pairs(case)}
    if op == "paged":
        hq, b = case["hq"], case["batch"]
        return {"bytes": 2 * sum(lens) * hkv * d * e + b * hq * (d * (e + 4) + 4) + 4 * sum(-(-x // case["page"]) for x in lens),
                "flops": 4 * d * hq * sum(lens)}
    if op == "append":
        return {"bytes": 4 * sum(new) * hkv * d * e, "flops": 0}
    row = 4 * hkv * d * e * case["layers"]  # one position's K and V in every layer, read and written
    if op == "fork":
        gone, parents = _fork_plan(case)
        n_pages, rows = _pages(case, new, 0.5)
        ints = 4 * (sum(len(rows[b]) for b in gone) * 2 + sum(len(rows[b]) for b in parents) * 3 + n_pages + 3 * case["batch"])
        return {"bytes": row * sum(new[b] % case["page"] for b in parents) + ints, "flops": 0}
    n_pages, rows = _pages(case, new, case["spare"])
    live = sum(len(x) for x in rows)
    return {"bytes": row * case["page"] * sum(x >= live for y in rows for x in y) + 4 * (2 * n_pages + 2 * live), "flops": 0}


# ------------------------------------------------------------------ inputs

class State:
    pass


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _keys(g, k, u):
    """Every hundredth key leans towards a direction that the queries share."""
    hit = torch.rand(k.shape[:-1], generator=g, device="cuda") < 0.01
    k += (3.0 * hit)[..., None].to(k.dtype) * u
    return k


def prepare(case, seed):
    s = State()
    s.case, op, d, hkv = dict(case), case["op"], case["d"], case["hkv"]
    g = _gen(seed)
    new, lens = _lens(case)
    dtype = DTYPES[case.get("dtype", "bf16")]
    u = torch.nn.functional.normalize(_randn(g, (d,), torch.float32), dim=0).to(dtype)
    if op == "prefill":
        s.q = _randn(g, (sum(new), case["hq"], d), dtype) + 2.0 * u
        s.k = _keys(g, _randn(g, (sum(lens), hkv, d), dtype), u)
        s.v = _randn(g, (sum(lens), hkv, d), dtype)
        s.cu_q, s.cu_k = (_ints([sum(x[:i]) for i in range(len(x) + 1)]) for x in (new, lens))
        s.max_q, s.max_k = max(new), max(lens)
        if own:
            import slow_sparse_kv_gb300 as sfi
            s.lay = sfi.PackedLayout(case["hq"], hkv, d, dtype, s.cu_q, s.cu_k, sum(new), sum(lens))
            s.out, s.lse = torch.empty_like(s.q), torch.empty(sum(new), case["hq"], device="cuda")
            s.ws = sfi.prefill_workspace(s.lay)
        return s
    spare = {"fork": 0.5, "compact": case.get("spare")}.get(op, 0.1)
    s.page = case["page"]
    s.n_pages, rows = _pages(case, lens, spare)
    s.width = max(len(r) for r in rows) + 1
    s.table = _ints([r + [-1] * (s.width - len(r)) for r in rows])
    s.len = _ints(lens)
    pool = (case.get("layers", 1), s.n_pages, hkv, s.page, d)
    s.k, s.v = _randn(g, pool, dtype), _randn(g, pool, dtype)
    if op == "paged":
        s.k, s.v = _keys(g, s.k, u)[0], s.v[0]
        s.q = _randn(g, (case["batch"], case["hq"], d), dtype) + 2.0 * u
    elif op == "append":
        s.k, s.v = s.k[0], s.v[0]
        s.k_new, s.v_new = _randn(g, (sum(new), hkv, d), dtype), _randn(g, (sum(new), hkv, d), dtype)
        s.cu = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    else:
        ref = [0] * s.n_pages
        for r in rows:
            for x in r:
                ref[x] += 1
        s.ref = _ints(ref)
        s.kept = (s.table.clone(), s.len.clone(), s.ref.clone())
        if op == "fork":
            s.gone, s.parents = _fork_plan(case)
            s.one = _ints([1] * case["batch"])
    if own:
        import slow_sparse_kv_gb300 as sfi
        s.lay = sfi.PagedLayout(case.get("hq", hkv), hkv, d, dtype, s.page, s.n_pages, s.table, s.len)
        s.ws = sfi.paged_workspace(s.lay)
        if op == "paged":
            s.out = torch.empty(case["batch"], case["hq"], d, device="cuda")
            s.lse = torch.empty(case["batch"], case["hq"], device="cuda")
        elif op != "append":
            s.store = sfi.PageStore(s.ref, s.k, s.v)
    return s


# --------------------------------------------------------------------- run

def run(s):
    return (_own if own else _plain)[s.case["op"]](s)


def _softmax_av(score, hidden, v):
    """softmax(score) v and the row's log-sum, with `hidden` places left out; a row without any gives 0 and -inf."""
    score.masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    base = top.masked_fill(top == -math.inf, 0.0)
    score.sub_(base).exp_()
    total = score.sum(-1, keepdim=True)
    lse = (base + total.log()).squeeze(-1)
    shape = score.shape
    out = (score.reshape(*shape[:2], -1, shape[-1]) @ v).reshape(*shape[:-1], v.shape[-1])
    return out / total.masked_fill(total == 0, 1.0), lse


def _plain_prefill(s):
    hq, hkv, d = s.case["hq"], s.case["hkv"], s.case["d"]
    cq, ck = s.cu_q.long(), s.cu_k.long()
    nq, nk = cq.diff(), ck.diff()
    i, j = torch.arange(s.max_q, device="cuda"), torch.arange(s.max_k, device="cuda")
    at_q = (cq[:-1, None] + i).clamp_max(s.q.shape[0] - 1)
    at_k = (ck[:-1, None] + j).clamp_max(s.k.shape[0] - 1)
    q = s.q[at_q].float().view(-1, s.max_q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    k, v = (x[at_k].float().transpose(1, 2) for x in (s.k, s.v))
    b = q.shape[0]
    score = q.reshape(b, hkv, -1, d) @ k.transpose(2, 3)
    score.mul_(1.0 / math.sqrt(d))
    hidden = (j > (i[:, None] + (nk - nq)[:, None, None])) | (j >= nk[:, None, None])
    o, lse = _softmax_av(score.view(b, hkv, hq // hkv, s.max_q, s.max_k), hidden[:, None, None], v)
    there = i < nq[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(b, s.max_q, hq, d)[there]
    return {"out": out.to(s.q.dtype), "lse": lse.permute(0, 3, 1, 2).reshape(b, s.max_q, hq)[there]}


def _plain_paged(s):
    hq, hkv, d = s.case["hq"], s.case["hkv"], s.case["d"]
    tab = s.table.long().clamp_min(0)
    b, w = tab.shape
    k, v = (x[tab].transpose(1, 2).reshape(b, hkv, w * s.page, d).float() for x in (s.k, s.v))
    score = s.q.float().view(b, hkv, hq // hkv, d) @ k.transpose(2, 3)
    score.mul_(1.0 / math.sqrt(d))
    hidden = torch.arange(w * s.page, device="cuda") >= s.len[:, None]
    o, lse = _softmax_av(score, hidden[:, None, None], v)
    return {"out": o.reshape(b, hq, d), "lse": lse.reshape(b, hq)}


def _plain_append(s):
    cu = s.cu.long()
    new = cu.diff()
    t = torch.arange(s.k_new.shape[0], device="cuda")
    b = torch.bucketize(t, cu[1:], right=True)
    pos = s.len.long()[b] - new[b] + t - cu[b]
    page = s.table.long()[b, pos // s.page]
    s.k[page, :, pos % s.page] = s.k_new
    s.v[page, :, pos % s.page] = s.v_new
    return {"k": s.k, "v": s.v}


def _restore(s):
    for x, y in zip((s.table, s.len, s.ref), s.kept):
        x.copy_(y)


def _plain_fork(s):
    _restore(s)
    p, width = s.page, s.width
    at = torch.arange(width, device="cuda")
    gone, parents = torch.tensor(s.gone, device="cuda"), torch.tensor(s.parents, device="cuda")
    # finished sequences give their pages back
    rows = s.table[gone]
    held = at < -(-s.len[gone] // p)[:, None]
    s.ref.index_add_(0, rows[held].long(), torch.full_like(rows[held], -1))
    s.table[gone] = torch.where(held, -1, rows)
    s.len[gone] = 0
    # forks share the full pages and get a copy of the last, partly filled one
    n = s.len[parents]
    full = (n // p)[:, None]
    rows = s.table[parents]
    shared = at < full
    s.ref.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    part = n % p > 0
    fresh = torch.nonzero(s.ref == 0).flatten()[:int(part.sum())]
    s.ref[fresh] = 1
    last = rows.gather(1, full.clamp_max(width - 1).long())[part, 0].long()
    row = torch.arange(p, device="cuda")
    used = (row < (n % p)[part][:, None])[:, None, :, None]
    for x in (s.k, s.v):
        x[:, fresh] = torch.where(used, x[:, last], x[:, fresh])
    mine = torch.where(shared, rows, s.table[gone])
    mine[part] = mine[part].scatter(1, full[part].long(), fresh.int()[:, None])
    s.table[gone] = mine
    s.len[gone] = n
    # every sequence grows by a token
    want = s.len % p == 0
    fresh = torch.nonzero(s.ref == 0).flatten()[:int(want.sum())]
    s.ref[fresh] = 1
    s.table[want] = s.table[want].scatter(1, (s.len[want] // p).long()[:, None], fresh.int()[:, None])
    s.len += s.one
    return {"k": s.k, "v": s.v, "table": s.table, "len": s.len, "ref": s.ref}


def _plain_compact(s):
    _restore(s)
    live = int((s.ref > 0).sum())
    holes = torch.nonzero(s.ref[:live] == 0).flatten()
    moved = torch.nonzero(s.ref[live:] > 0).flatten() + live
    for x in (s.k, s.v):
        x[:, holes] = x[:, moved]
    to = torch.arange(s.n_pages, device="cuda", dtype=torch.int32)
    to[moved] = holes.int()
    held = torch.arange(s.width, device="cuda") < -(-s.len // s.page)[:, None]
    s.table.copy_(torch.where(held, to[s.table.long().clamp_min(0)], s.table))
    s.ref[holes] = s.ref[moved]
    s.ref[live:] = 0
    return {"k": s.k, "v": s.v, "table": s.table, "len": s.len, "ref": s.ref}


_plain = {"prefill": _plain_prefill, "paged": _plain_paged, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}


def _own_prefill(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_prefill_attn(s.lay, s.q, s.k, s.v, s.out, s.lse, s.ws)
    return {"out": s.out, "lse": s.lse}


def _own_paged(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_paged_attn(s.lay, s.q, s.k, s.v, s.out, s.lse, s.ws)
    return {"out": s.out, "lse": s.lse}


def _own_append(s):
    import slow_sparse_kv_gb300 as sfi
    sfi.sfi_paged_append(s.lay, s.k_new, s.v_new, s.k, s.v, s.cu, s.ws)
    return {"k": s.k, "v": s.v}


def _own_fork(s):
    import slow_sparse_kv_gb300 as sfi
    _restore(s)
    sfi.sfi_pages_free(s.lay, s.store, s.gone, s.ws)
    sfi.sfi_pages_fork(s.lay, s.store, s.parents, s.gone, s.ws)
    sfi.sfi_pages_extend(s.lay, s.store, s.one, s.ws)
    return {"k": s.k, "v": s.v, "table": s.table, "len": s.len, "ref": s.ref}


def _own_compact(s):
    import slow_sparse_kv_gb300 as sfi
    _restore(s)
    sfi.sfi_pages_compact(s.lay, s.store, None, s.ws)
    return {"k": s.k, "v": s.v, "table": s.table, "len": s.len, "ref": s.ref}


_own = {"prefill": _own_prefill, "paged": _own_paged, "append": _own_append, "fork": _own_fork, "compact": _own_compact}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """Attention from its definition, one sequence and KV head at a time, in 64 bits; the other operators move
    values without computing any."""
    if case["op"] not in ("prefill", "paged"):
        return None
    s = prepare(case, seed)
    new, lens = _lens(case)
    group, d = case["hq"] // case["hkv"], case["d"]
    out, lse = [], []
    for b in range(case["batch"]):
        for h in range(case["hkv"]):
            heads = slice(h * group, (h + 1) * group)
            if case["op"] == "prefill":
                at = sum(lens[:b])
                k, v = s.k[at:at + lens[b], h].double(), s.v[at:at + lens[b], h].double()
                q = s.q[sum(new[:b]):sum(new[:b + 1]), heads].double()
            else:
                ids = s.table[b, :-(-lens[b] // s.page)].long()
                k, v = (x[ids, h].reshape(-1, d)[:lens[b]].double() for x in (s.k, s.v))
                q = s.q[b:b + 1, heads].double()
            o, z = [], []
            for i in range(0, q.shape[0], 2048):  # rows i.. see the keys up to their own position
                rows = min(2048, q.shape[0] - i)
                end = lens[b] - q.shape[0] + i + rows
                t = torch.einsum("rgd,kd->rgk", q[i:i + rows], k[:end]) / d ** 0.5
                t += torch.full((rows, end), -math.inf, dtype=torch.float64, device="cuda").triu_(end - rows + 1)[:, None]
                z.append(torch.logsumexp(t, -1))
                o.append(torch.exp(t - z[-1][..., None]) @ v[:end])
            out.append(torch.cat(o))
            lse.append(torch.cat(z))
    n = case["hkv"]
    out = torch.cat([torch.cat(out[i:i + n], 1) for i in range(0, len(out), n)])
    lse = torch.cat([torch.cat(lse[i:i + n], 1) for i in range(0, len(lse), n)])
    return {"out": out, "lse": lse}
