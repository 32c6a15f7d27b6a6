"""A paged cache in 8 bits (sfi_paged_append_q8, sfi_paged_attn_q8, the bookkeeping on such pools)
against the 64-bit restatements."""
import numpy as np
import pytest
import torch

import oracle.heads_oracle as H
import oracle.paged_oracle as P
from tests.paged_testlib import close, close_lse, f32_tolerance, f64, ints, normal, offsets, pool_of
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16, F32, I8, E4M3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
FMT = {I8: "i8", E4M3: "e4m3"}


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def noise(shape, seed):
    """Bytes of all kinds, NaN codes and scales among them."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()


def values(lay, pool):
    """What a pool's rows stand for, in 64 bits."""
    return f64(lay.codes(pool).float()) * f64(lay.scales(pool))[..., None]


class Cache:
    """Pools whose rows are normal numbers of very different sizes; `hkv` pools of noise elsewhere."""

    def __init__(self, sfi, hq, hkv, d, fmt, page, lens, seed=1, gap=0, spread=1.0):
        self.hq, self.hkv, self.d, self.fmt, self.page, self.lens = hq, hkv, d, fmt, page, list(lens)
        self.n_pages, self.rows = pool_of(lens, page, 3, seed)
        self.table, self.len = ints(self.rows.tolist()), ints(self.lens)
        size = -(-hkv * page * (d + 4) // 16) * 16
        self.lay = sfi.PagedLayout(hq, hkv, d, fmt, page, self.n_pages, self.table, self.len, page_stride=(size + gap) if gap else 0)
        assert self.lay.page_bytes == size
        self.k, self.v = (noise((self.n_pages, size + gap), seed + i)[:, :size] for i in (5, 6))
        g = torch.Generator().manual_seed(seed + 7)
        for pool in (self.k, self.v):
            x = torch.randn(self.n_pages, hkv, page, d, generator=g)
            x *= torch.exp2(spread * torch.randn(self.n_pages, hkv, page, 1, generator=g))
            codes, scales = H.quantise(x.numpy(), FMT[fmt])
            self.lay.codes(pool).copy_(torch.from_numpy(codes).float().to(fmt))
            self.lay.scales(pool).copy_(torch.from_numpy(scales))

    def spoil(self, seed=99):
        """Noise in every row that no sequence holds."""
        used = torch.zeros(self.n_pages, self.page, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for i in range(n):
                used[self.rows[b, i // self.page], i % self.page] = True
        for i, pool in enumerate((self.k, self.v)):
            junk = noise(pool.shape, seed + i)
            for of in (self.lay.codes, self.lay.scales):
                there = of(pool)
                keep = used.cuda()[:, None, :].expand(there.shape[:3])
                raw, new = (t.view(torch.uint8) if t.dtype == E4M3 else t for t in (there, of(junk)))
                raw.copy_(torch.where(keep[..., None] if raw.dim() == 4 else keep, raw, new))

    def run(self, sfi, q, status=0, ws=None):
        ws = sfi.paged_workspace(self.lay) if ws is None else ws
        out = torch.full((len(self.lens), self.hq, self.d), 7.0, device="cuda")
        lse = torch.full((len(self.lens), self.hq), 7.0, device="cuda")
        sfi.sfi_paged_attn_q8(self.lay, q, self.k, self.v, out, lse, ws)
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == status
        return out, lse

    def check(self, q, out, lse):
        v = values(self.lay, self.v)
        held = np.concatenate([np.zeros(0)] + [np.abs(v[self.rows[b, i // self.page], :, i % self.page]).ravel()
                                               for b, n in enumerate(self.lens) for i in range(n)])
        ref, rl, scale, size = P.paged(f64(q), values(self.lay, self.k), v, self.rows, self.lens)
        close(f64(out), ref, tolerance(ref, scale, size, self.d, max(self.lens), q.dtype, held.max(initial=0.0)), "out")
        # (three products of a score with its factors, and fp32 queries in 22 bits)
        close_lse(f64(lse), rl, size * (1 + (2.0 ** -21 if q.dtype == F32 else 0) / (2.0 ** -23 * self.d)), self.d + 8)


def tolerance(ref, scale, size, d, n, dtype, top):
    """Elementwise bound: that of an fp32 attention (scores with 8 roundings more: factors and scales),
    queries in two fp16 terms where they are fp32 (2^-21 with both roundings), p in two terms
    (2^-11 each), and of what these drop below their smallest number, 2^-25 on a scale on
    which the tile's largest p sv counts as 2^14 at least, p being at most 2^4: 2^-35
    of the largest value for each of n positions."""
    if dtype == F32:
        size = size * (1 + 2.0 ** -21 / (2.0 ** -23 * d))
    return f32_tolerance(ref, scale, size, d + 8, n, False) + 2.0 ** -22 * scale + n * 2.0 ** -35 * top


CASES = [
    # (H_q, H_kv, d, format, type of q, page size, lengths)
    (8, 2, 128, I8, BF16, 16, [1]),
    (8, 2, 128, E4M3, BF16, 16, [0, 15, 16, 17, 0, 300]),
    (8, 2, 64, I8, F32, 32, [700, 31, 32, 33, 64]),
    (4, 4, 128, E4M3, F32, 48, [500, 47, 49]),
    (8, 1, 128, I8, BF16, 64, [2100]),
    (16, 1, 128, I8, F32, 16, [130, 1]),
    (16, 2, 64, E4M3, F32, 80, [330, 81]),
    (10, 1, 64, E4M3, BF16, 256, [800, 255]),
    (3, 1, 128, I8, BF16, 1024, [77, 1025]),
    (14, 2, 128, E4M3, BF16, 1, [40, 7]),        # pages gathered row by row
    (8, 2, 128, I8, F32, 5, [203, 4, 0]),
    (6, 2, 64, E4M3, BF16, 24, [100, 24, 25]),
    (16, 1, 64, I8, BF16, 20, [333]),
    (16, 1, 128, E4M3, BF16, 40, [333, 95]),
    (5, 5, 64, I8, F32, 3, [101, 0]),
    (1, 1, 64, E4M3, F32, 7, [29]),
]


@pytest.mark.parametrize("hq,hkv,d,fmt,dtype,page,lens", CASES)
def test_attn_matches_oracle(sfi, hq, hkv, d, fmt, dtype, page, lens):
    c = Cache(sfi, hq, hkv, d, fmt, page, lens)
    q = normal((len(lens), hq, d), dtype, 11)
    out, lse = c.run(sfi, q)
    c.check(q, out, lse)
    again, lse2 = c.run(sfi, q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    c.spoil()
    again, lse2 = c.run(sfi, q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("fmt,page,gap", [(I8, 16, 48), (E4M3, 12, 16), (I8, 64, 4096)])
def test_pages_apart(sfi, fmt, page, gap):
    c = Cache(sfi, 4, 2, 64, fmt, page, [90, 33], gap=gap)
    q = normal((2, 4, 64), BF16, 12)
    c.check(q, *c.run(sfi, q))


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_of_all_sizes(sfi, fmt, dtype):
    """Rows from 2^-20 to 2^20 beside each other, queries from 2^-10 to 2^10, rows of zeros."""
    c = Cache(sfi, 4, 1, 128, fmt, 16, [400, 33], spread=5.0)
    for pool in (c.k, c.v):
        c.lay.codes(pool).view(torch.uint8)[c.rows[0, 2], 0, 3] = 0
        c.lay.scales(pool)[c.rows[0, 2], 0, 3] = 0
    q = (normal((2, 4, 128), F32, 13) * torch.exp2(torch.tensor([-10.0, -3.0, 0.0, -6.0], device="cuda"))[None, :, None] * 2.0 ** -5).to(dtype)
    q[1, 0] = 0
    q[1, 1, 1:] = 0
    c.check(q, *c.run(sfi, q))
    # a pool of tiny values, and one of large ones
    for up in (2.0 ** -70, 2.0 ** 60):
        c.lay.scales(c.v).mul_(up)
        c.check(q, *c.run(sfi, q))


@pytest.mark.parametrize("fmt,dtype", [(I8, BF16), (E4M3, F32)])
@pytest.mark.parametrize("up", [90, -90])
def test_large_keys_and_small_queries(sfi, fmt, dtype, up):
    """And the other way round: scores of the usual size."""
    c = Cache(sfi, 4, 2, 128, fmt, 16, [200, 33])
    c.lay.scales(c.k).mul_(2.0 ** up)
    q = (normal((2, 4, 128), F32, 22) * 2.0 ** -up).to(dtype)
    c.check(q, *c.run(sfi, q))


@pytest.mark.parametrize("up", [20, 40])
@pytest.mark.parametrize("fmt,dtype", [(I8, BF16), (E4M3, F32)])
def test_large_values_that_a_head_leaves_out(sfi, fmt, dtype, up):
    """A position in every tile whose value is 2^up times the others', which the one head of its
    group leaves out (a score of about -80) and the other attends to alone."""
    lens = [400, 33]
    c = Cache(sfi, 4, 2, 128, fmt, 16, lens, spread=0.0)
    q = normal((2, 4, 128), dtype, 21)
    q[:, 1::2] = -q[:, ::2]
    for b, n in enumerate(lens):
        for i in range(3, n, 32):
            for g in range(2):
                at = (int(c.rows[b, i // 16]), g, i % 16)
                x = q[b, 2 * g].float()
                c.lay.codes(c.k)[at] = (-40 * torch.sign(x)).to(fmt)
                c.lay.scales(c.k)[at] = 80 * 128 ** 0.5 / 40 / float(x.abs().sum())
                c.lay.scales(c.v)[at] *= 2.0 ** up
    out, lse = c.run(sfi, q)
    ref, rl, scale, size = P.paged(f64(q), values(c.lay, c.k), values(c.lay, c.v), c.rows, lens)
    # (as in `tolerance`, but what p in two terms drops is 2^-39 of the largest p sv of a tile and head
    # for each position; times a code, which is at most twice its row's largest)
    tol = tolerance(ref, scale, size, 128, 400, dtype, 0.0) + 400 * 2.0 ** -38 * scale.max(-1, keepdims=True)
    close(f64(out), ref, tol, "out")
    close_lse(f64(lse), rl, size * (1 + 2.0 ** -21 / (2.0 ** -23 * 128)), 128 + 8)


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_growing_scores_rescale(sfi, fmt):
    c = Cache(sfi, 4, 1, 128, fmt, 16, [1500], spread=0.0)
    ramp = torch.linspace(0.1, 6.0, 94, device="cuda")
    c.lay.scales(c.k)[c.rows[0, :94].tolist()] *= ramp[:, None, None]
    q = normal((1, 4, 128), BF16, 14)
    c.check(q, *c.run(sfi, q))


@pytest.mark.parametrize("fmt", [I8, E4M3])
def test_nan_scale_reaches_its_sequence_and_head_only(sfi, fmt):
    c = Cache(sfi, 4, 2, 64, fmt, 16, [50, 40, 60])
    q = normal((3, 4, 64), BF16, 15)
    good, gl = c.run(sfi, q)
    for pool, lse_bad in ((c.v, False), (c.k, True)):
        at = (int(c.rows[1, 1]), 1, 5)  # position 21 of sequence 1, KV head 1
        keep = float(c.lay.scales(pool)[at])
        c.lay.scales(pool)[at] = float("nan")
        out, lse = c.run(sfi, q)
        assert out[1, 2:].isnan().all() and lse[1, 2:].isnan().all() == lse_bad
        rest = torch.ones(3, 4, dtype=torch.bool, device="cuda")
        rest[1, 2:] = False
        assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], gl[rest])
        c.lay.scales(pool)[at] = keep


def test_bad_pages_and_lengths(sfi):
    c = Cache(sfi, 4, 2, 64, I8, 16, [50, 40])
    q = normal((2, 4, 64), BF16, 16)
    good, _ = c.run(sfi, q)
    for bad in (-3, c.n_pages, 1 << 30):
        c.table[0, 1] = bad
        out, _ = c.run(sfi, q, status=sfi.SFI_DEV_BAD_INDEX)
        assert torch.equal(out[1], good[1])
    c.table[0, 1] = int(c.rows[0, 1])
    c.len[0] = -4
    out, lse = c.run(sfi, q, status=sfi.SFI_DEV_LEN_OVER_CAP)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.equal(out[1], good[1])


@pytest.mark.parametrize("fmt,dtype,page", [(I8, BF16, 32), (E4M3, F32, 16), (I8, F32, 20)])
def test_wait_limit(sfi, fmt, dtype, page):
    """A one-clock limit: the waits give up, the status says so, nothing is left in flight.  The
    cache is larger than L2, so that some wait is always early."""
    n, hq, hkv, d = 16384, 8, 2, 128
    per = -(-n // page)
    n_pages = 64 * per
    table = torch.randperm(n_pages, device="cuda").view(64, per).int()
    lay = sfi.PagedLayout(hq, hkv, d, fmt, page, n_pages, table, ints([n] * 64))
    k, v = (torch.zeros(n_pages, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    for pool in (k, v):
        lay.codes(pool).view(torch.uint8).copy_(torch.randint(0, 100, (1, hkv, page, d), device="cuda", dtype=torch.uint8))
        lay.scales(pool).fill_(0.01)
    q = normal((64, hq, d), dtype, 1)
    ws, good, out = sfi.paged_workspace(lay), *(torch.empty(64, hq, d, device="cuda") for _ in range(2))
    sfi.sfi_paged_attn_q8(lay, q, k, v, good, None, ws)
    assert sfi.sfi_read_status(ws) == 0
    sfi.lib.sfi_set_wait_limit(1)
    try:
        for _ in range(2):
            sfi.sfi_paged_attn_q8(lay, q, k, v, out, None, ws)
            assert sfi.sfi_read_status(ws) == sfi.SFI_DEV_WAIT_TIMEOUT
    finally:
        sfi.lib.sfi_set_wait_limit(0)
    ws.zero_()
    sfi.sfi_paged_attn_q8(lay, q, k, v, out, None, ws)
    assert sfi.sfi_read_status(ws) == 0 and torch.equal(good, out)


@pytest.mark.parametrize("fmt,dtype,lens,page", [(I8, BF16, [(i * 7) % 41 for i in range(300)], 16), (E4M3, F32, [1 + i % 3 for i in range(1024)], 20)])
def test_many_sequences(sfi, fmt, dtype, lens, page):
    c = Cache(sfi, 4, 2, 64, fmt, page, lens)
    q = normal((len(lens), 4, 64), dtype, 17)
    c.check(q, *c.run(sfi, q))


@pytest.mark.parametrize("hq,hkv,d,fmt,page,lens", [
    (4, 2, 64, I8, 16, [70000, 8191, 0, 130001]), (32, 8, 64, E4M3, 20, [24001] * 4), (8, 8, 128, I8, 64, [24576] * 12),
    (8, 2, 128, E4M3, 16, [200000, 160001, 0, 280000]),
])
def test_long_units_are_cut_and_joined(sfi, hq, hkv, d, fmt, page, lens):
    n_pages, rows = pool_of(lens, page, 3, 60)
    table, ln = ints(rows.tolist()), ints(lens)
    lay = sfi.PagedLayout(hq, hkv, d, fmt, page, n_pages, table, ln)
    g = torch.Generator(device="cuda").manual_seed(61)
    k, v = (torch.zeros(n_pages, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    for pool in (k, v):
        lay.codes(pool).copy_(torch.randint(-127, 128, lay.codes(pool).shape, generator=g, device="cuda").float().to(fmt))
        lay.scales(pool).copy_(torch.rand(lay.scales(pool).shape, generator=g, device="cuda") * 0.02 + 0.001)
    q = normal((len(lens), hq, d), BF16, 62)
    out, lse = torch.empty(len(lens), hq, d, device="cuda"), torch.empty(len(lens), hq, device="cuda")
    ws = sfi.paged_workspace(lay)
    sfi.sfi_paged_attn_q8(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    sfi.sfi_paged_attn_q8(lay, q, k, v, out2, lse2, ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    G = hq // hkv
    for b in sorted({0, len(lens) // 2, len(lens) - 1}):
        ids = rows[b][:-(-lens[b] // page)].tolist()
        for h in sorted({0, hkv - 1}):
            K, V = (f64(lay.codes(x)[:, h].view(torch.uint8)[ids].view(fmt).float()) * f64(lay.scales(x)[ids, h])[..., None] for x in (k, v))
            K, V = (x.reshape(-1, d)[:lens[b]] for x in (K, V))
            for e in sorted({0, G - 1}):
                if lens[b] == 0:
                    assert (out[b] == 0).all()
                    continue
                ref, rl, scale, size = P.attend(f64(q[b, h * G + e]), K, V, lens[b])
                tol = tolerance(ref[None], scale[None], np.array([size]), d, lens[b], BF16, np.abs(V).max())[0]
                close(f64(out[b, h * G + e]), ref, tol, "out")
                close_lse(f64(lse[b, h * G + e])[None], np.array([rl]), np.array([size]), d + 8)


def test_pool_beyond_4_gb(sfi):
    """Pages far apart: offsets of codes and scales beyond 2^32 bytes, with boxes and gathered."""
    for page in (16, 12):
        stride = (1 << 31) + 16
        lay_len, table = ints([2 * page + 5]), ints([[2, 0, 1, -1]])
        lay = sfi.PagedLayout(2, 1, 64, I8, page, 3, table, lay_len, page_stride=stride)
        k, v = (torch.zeros(2 * stride + lay.page_bytes, dtype=torch.uint8, device="cuda").as_strided((3, lay.page_bytes), (stride, 1)) for _ in range(2))
        new = [normal((2 * page + 5, 1, 64), F32, 20 + i) for i in range(2)]
        ws = sfi.paged_workspace(lay)
        sfi.sfi_paged_append_q8(lay, *new, k, v, ints([0, 2 * page + 5]), ws)
        q, out, lse = normal((1, 2, 64), BF16, 22), torch.empty(1, 2, 64, device="cuda"), torch.empty(1, 2, device="cuda")
        sfi.sfi_paged_attn_q8(lay, q, k, v, out, lse, ws)
        assert sfi.sfi_read_status(ws) == 0
        K, V = values(lay, k), values(lay, v)
        ref, rl, scale, size = P.paged(f64(q), K, V, [[2, 0, 1]], [2 * page + 5])
        close(f64(out), ref, tolerance(ref, scale, size, 64, 2 * page + 5, BF16, np.abs(V).max()), "out")
        del k, v
        torch.cuda.empty_cache()


# ------------------------------------------------------------------ storing

def special_rows(d, seed):
    """Rows where rounding is hard: ties (half of the maximum is one), all powers of two, maxima at
    448 and just above, zeros, tiny and subnormal numbers, huge ones, infinities and NaN."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(40, 1, d, generator=g)
    x[0] = 0
    x[1, 0, :8] = torch.tensor([2.0, 1.0, -1.0, 0.5, 0.25, -0.125, 3.0, -4.0])
    x[2] = torch.arange(d).float() * 0.5
    x[3] = torch.arange(d).float() * (127.0 / (d - 1))
    x[4, 0] = 448.0 * torch.rand(d, generator=g)
    x[4, 0, 0] = 448.0
    x[5] = x[4]
    x[5, 0, 0] = 450.0
    x[6] *= 1e-30
    x[7] *= 1e-38
    x[8] *= 1e-40
    x[9] *= 1e-44
    x[10] *= 1e37
    x[11, 0, 3] = 3.3e38
    x[12, 0, 3] = float("inf")
    x[13, 0, 3] = float("nan")
    x[14, 0, d - 1] = -float("inf")
    for i in range(15, 40):  # multiples of half a step of the row's own scale
        top = float(torch.randint(1, 255, (1,), generator=g)) * 2.0 ** (i - 25)
        x[i, 0] = torch.randint(-254, 255, (d,), generator=g).float() * (top / 254)
        x[i, 0, 0] = top
    return x


@pytest.mark.parametrize("fmt", [I8, E4M3])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,hkv,page", [(64, 3, 16), (128, 2, 5), (128, 9, 32)])
def test_append_stores_the_exact_codes(sfi, fmt, dtype, d, hkv, page):
    lens, new = [300, 90, 0, 41, 7], [290, 1, 0, 40, 7]
    n_pages, rows = pool_of(lens, page, 2, 3)
    lay = sfi.PagedLayout(hkv, hkv, d, fmt, page, n_pages, ints(rows.tolist()), ints(lens))
    total = sum(new)
    joint = torch.zeros(total, 3 * hkv, d)
    x = torch.cat([special_rows(d, 1 + i) for i in range(-(-total * 2 * hkv // 40))]).reshape(-1, d)
    joint[:, hkv:] = x[:total * 2 * hkv].reshape(total, 2 * hkv, d)
    joint = joint.to(dtype).cuda()
    k_new, v_new = joint[:, hkv:2 * hkv], joint[:, 2 * hkv:]  # slices of a joint projection
    k, v = noise((n_pages, lay.page_bytes), 4), noise((n_pages, lay.page_bytes), 5)
    before = [x.cpu().clone() for x in (k, v)]
    ws = sfi.paged_workspace(lay)
    sfi.sfi_paged_append_q8(lay, k_new, v_new, k, v, ints(offsets(new)), ws)
    assert sfi.sfi_read_status(ws) == 0
    for rows_new, pool, was in ((k_new, k, before[0]), (v_new, v, before[1])):
        codes, scales = H.quantise(rows_new.float().cpu().numpy(), FMT[fmt])
        want = was.clone()
        wc, wsc = lay.codes(want), lay.scales(want)
        for b, m in enumerate(new):
            for i in range(m):
                pos, t = lens[b] - m + i, offsets(new)[b] + i
                page_id = int(rows[b, pos // page])
                wc[page_id, :, pos % page] = torch.from_numpy(codes[t]).float().to(fmt)
                wsc[page_id, :, pos % page] = torch.from_numpy(scales[t])
        got = pool.cpu()
        # negative zero is a code of e4m3 (and the NaN scales' bits are not compared)
        gc, gs = lay.codes(got), lay.scales(got)
        if fmt == E4M3:
            same = (gc.view(torch.uint8) == wc.view(torch.uint8)) | ((gc.float() == 0) & (wc.float() == 0))
        else:
            same = gc == wc
        assert same.all(), (~same).nonzero()[:4]
        assert torch.equal(gs.isnan() | (gs == wsc), torch.ones_like(gs, dtype=torch.bool)) and torch.equal(gs.isnan(), wsc.isnan())
        tail = lay.n_kv_heads * page * (d + 4)
        assert torch.equal(got[:, tail:], was[:, tail:])


def test_int8_scales_are_rounded_quotients(sfi):
    """2^20 rows of fp32 whose largest elements go over the significands and the exponents of both ways to the
    scale, and of whose other elements one is half of that, next to a tie."""
    n, hkv, d, page = 1 << 17, 8, 64, 1024
    lay = sfi.PagedLayout(hkv, hkv, d, I8, page, n // page, ints([list(range(n // page))]), ints([n]))
    x = torch.zeros(n, hkv, d)
    at = torch.arange(n * hkv, dtype=torch.int64)
    bits = (at * 8 + at % 8) % (1 << 23) | (60 + at * 7 % 180) << 23
    top = bits.int().view(torch.float32).view(n, hkv)
    x[..., 5], x[..., 9] = top, -0.5 * top
    k, v = (torch.zeros(n // page, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    ws = sfi.paged_workspace(lay)
    sfi.sfi_paged_append_q8(lay, x.cuda(), -x.cuda(), k, v, ints([0, n]), ws)
    assert sfi.sfi_read_status(ws) == 0
    scale = torch.from_numpy(top.numpy() / np.float32(127))
    half = torch.from_numpy(np.rint(0.5 * top.numpy().astype(np.float64) / scale.numpy())).to(I8)
    for pool, sign in ((k, 1), (v, -1)):
        codes, scales = (t.cpu().transpose(1, 2).flatten(0, 1) for t in (lay.codes(pool), lay.scales(pool)))
        assert torch.equal(scales, scale)
        assert (codes[..., 5] == sign * 127).all() and torch.equal(codes[..., 9], -sign * half)


def test_append_one_row_each_and_idle_slots(sfi):
    lens = [5, 0, 33, 16]
    n_pages, rows = pool_of(lens, 16, 2, 7)
    lay = sfi.PagedLayout(2, 2, 64, E4M3, 16, n_pages, ints(rows.tolist()), ints(lens))
    k, v = (torch.zeros(n_pages, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    new = [normal((4, 2, 64), BF16, 30 + i) for i in range(2)]
    ws = sfi.paged_workspace(lay)
    sfi.sfi_paged_append_q8(lay, *new, k, v, None, ws)
    assert sfi.sfi_read_status(ws) == 0
    for x, pool in zip(new, (k, v)):
        codes, scales = H.quantise(x.float().cpu().numpy(), "e4m3")
        got = values(lay, pool)
        for b, n in enumerate(lens):
            if n:
                at = (int(rows[b, (n - 1) // 16]), slice(None), (n - 1) % 16)
                assert np.array_equal(got[at], codes[b] * scales[b][..., None])
                got[at] = 0
        assert (got == 0).all()


def test_append_flags(sfi):
    """Rows that leave the sequence or the pool are left out and flagged, the others stored."""
    lens = [20, 30]
    n_pages, rows = pool_of(lens, 16, 2, 8)
    table, ln = ints(rows.tolist()), ints(lens)
    lay = sfi.PagedLayout(1, 1, 64, I8, 16, n_pages, table, ln)
    new = [normal((50, 1, 64), F32, 40 + i) for i in range(2)]
    for what, flag in (("page", sfi.SFI_DEV_BAD_INDEX), ("len", sfi.SFI_DEV_LEN_OVER_CAP), ("more", sfi.SFI_DEV_LEN_OVER_CAP)):
        k, v = (torch.zeros(n_pages, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
        ws = sfi.paged_workspace(lay)
        cu = [0, 20, 50]
        if what == "page":
            table[0, 0] = n_pages
        elif what == "len":
            ln[0] = -1
        else:
            cu = [0, 21, 50]
        sfi.sfi_paged_append_q8(lay, *new, k, v, ints(cu), ws)
        assert sfi.sfi_read_status(ws) == flag
        table[0, 0], ln[0] = int(rows[0, 0]), 20
        first = lay.scales(k)[rows[0, 0].item()]
        assert (first == 0).all(), what
        if what != "more":
            assert (lay.scales(k)[rows[1, 0].item()] > 0).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,page,d", [(I8, 16, 128), (E4M3, 5, 64), (I8, 7, 128)])
def test_bookkeeping_moves_codes_and_scales(sfi, fmt, page, d):
    """Prompts in, forks, tokens, frees, a compaction, page copies: what each sequence reads is what it stored."""
    hkv, layers, B, n_pages = 3, 2, 6, 60
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    ln = torch.zeros(B, dtype=torch.int32, device="cuda")
    lay = sfi.PagedLayout(2 * hkv, hkv, d, fmt, page, n_pages, table, ln)
    k, v = noise((layers, n_pages, lay.page_bytes), 50), noise((layers, n_pages, lay.page_bytes), 51)
    store = sfi.PageStore(torch.zeros(n_pages, dtype=torch.int32, device="cuda"), k, v)
    ws = sfi.paged_workspace(lay)
    held = [[np.zeros((layers, 2, 0, hkv, d))][0] for _ in range(B)]
    seed = [60]

    def grow(new):
        sfi.sfi_pages_extend(lay, store, ints(new), ws)
        cu = offsets(new)
        for layer in range(layers):
            x = [normal((sum(new), hkv, d), BF16, seed[0] + i) for i in range(2)]
            seed[0] += 2
            sfi.sfi_paged_append_q8(lay, *x, k[layer], v[layer], ints(cu), ws)
            vals = []
            for t in x:
                c, s = H.quantise(t.float().cpu().numpy(), FMT[fmt])
                vals.append(c * s[..., None].astype(np.float64))
            for b in range(B):
                if new[b]:
                    add = np.stack([y[cu[b]:cu[b + 1]] for y in vals])
                    if layer == 0:
                        held[b] = np.concatenate([held[b], np.zeros((layers, 2, new[b], hkv, d))], 2)
                    held[b][layer, :, -new[b]:] = add
        torch.cuda.synchronize()

    def check():
        assert sfi.sfi_read_status(ws) == 0
        tab, lens = table.cpu().numpy(), ln.cpu().numpy()
        for layer in range(layers):
            K, V = values(lay, k[layer]), values(lay, v[layer])
            for b in range(B):
                assert lens[b] == held[b].shape[2]
                for i, pool in enumerate((K, V)):
                    got = [pool[tab[b, p // page], :, p % page] for p in range(lens[b])]
                    assert not got or np.array_equal(np.stack(got), held[b][layer, i]), (b, layer, i)
            q = normal((B, 2 * hkv, d), BF16, 90 + layer)
            out, lse = torch.empty(B, 2 * hkv, d, device="cuda"), torch.empty(B, 2 * hkv, device="cuda")
            sfi.sfi_paged_attn_q8(lay, q, k[layer], v[layer], out, lse, ws)
            K, V = (np.nan_to_num(x) for x in (K, V))
            ref, rl, scale, size = P.paged(f64(q), K, V, tab, lens)
            top = max([np.abs(h[layer]).max(initial=0.0) for h in held])
            close(f64(out), ref, tolerance(ref, scale, size, d, max(lens), BF16, top), "out")

    grow([2 * page + 3, page, 0, 1, 0, 0])
    check()
    sfi.sfi_pages_fork(lay, store, [0, 0, 1], [2, 4, 5], ws)
    for s, t in ((0, 2), (0, 4), (1, 5)):
        held[t] = held[s].copy()
    check()
    grow([1] * B)
    grow([0, 3, 5, page, 1, 2])
    check()
    sfi.sfi_pages_free(lay, store, [0, 3], ws)
    held[0] = held[3] = np.zeros((layers, 2, 0, hkv, d))
    check()
    sfi.sfi_pages_compact(lay, store, None, ws)
    check()
    # the first page of sequence 1 as a copy in a free place
    free = int((store.ref == 0).nonzero()[-1])
    sfi.sfi_pages_copy(lay, store, table[1, :1].contiguous(), ints([free]), ws)
    store.ref[int(table[1, 0])] -= 1
    store.ref[free] += 1
    table[1, 0] = free
    grow([0, 1, 1, 2, 0, 1])
    check()


def test_from_projection_to_attention(sfi):
    """A prompt and two tokens: norm and rotation, into the 8-bit cache, attention, all in one graph for the tokens."""
    hq, hkv, d, page = 8, 2, 128, 16
    lens = [37, 90]
    table = ints([[0, 2, 4, 6, 8, 10, 12], [1, 3, 5, 7, 9, 11, 13]])
    ln = ints(lens)
    lay = sfi.PagedLayout(hq, hkv, d, I8, page, 14, table, ln)
    k, v = (torch.zeros(14, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    ws = sfi.paged_workspace(lay)
    wq, wk = (1 + 0.1 * normal((d,), BF16, 70)), (1 + 0.1 * normal((d,), BF16, 71))

    def heads(x, pos):
        rot = sfi.RotaryLayout(hq, hkv, d, BF16, pos)
        qo, ko = torch.empty(x.shape[0], hq, d, dtype=BF16, device="cuda"), torch.empty(x.shape[0], hkv, d, dtype=BF16, device="cuda")
        return rot, qo, ko

    x = normal((sum(lens), hq + 2 * hkv, d), BF16, 72)
    rot, qo, ko = heads(x, ints(list(range(37)) + list(range(90))))
    sfi.sfi_qk_norm_rope(rot, x[:, :hq], x[:, hq:hq + hkv], qo, ko, wq, wk)
    sfi.sfi_paged_append_q8(lay, ko, x[:, hq + hkv:], k, v, ints(offsets(lens)), ws)
    # the tokens: positions are the lengths less one
    x1 = normal((2, hq + 2 * hkv, d), BF16, 73)
    rot = sfi.RotaryLayout(hq, hkv, d, BF16, ln, pos_offset=-1)
    q1, k1 = torch.empty(2, hq, d, dtype=BF16, device="cuda"), torch.empty(2, hkv, d, dtype=BF16, device="cuda")
    out, lse = torch.empty(2, hq, d, device="cuda"), torch.empty(2, hq, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ln.add_(1)
        sfi.sfi_qk_norm_rope(rot, x1[:, :hq], x1[:, hq:hq + hkv], q1, k1, wq, wk)
        sfi.sfi_paged_append_q8(lay, k1, x1[:, hq + hkv:], k, v, None, ws)
        sfi.sfi_paged_attn_q8(lay, q1, k, v, out, lse, ws)
    for step in range(2):
        x1.copy_(normal((2, hq + 2 * hkv, d), BF16, 74 + step))
        graph.replay()
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == 0
        now = [n + step + 1 for n in lens]
        assert ln.tolist() == now
        freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
        ref, size = H.norm_rope(f64(x1[:, :hq]), f64(wq), [n - 1 for n in now], freq, False, 1e-6)
        close(f64(q1), ref, size * 2.0 ** -19 * 1.01 + 2.0 ** -8 * np.abs(ref), "q")
        K, V = values(lay, k), values(lay, v)
        for b, n in enumerate(now):  # the token's own row, as it was stored
            c, s = H.quantise(k1[b].float().cpu().numpy(), "i8")
            assert np.array_equal(K[int(table[b, (n - 1) // page]), :, (n - 1) % page], c * s[..., None].astype(np.float64))
        ref, rl, scale, size = P.paged(f64(q1), K, V, table.cpu().numpy(), now)
        close(f64(out), ref, tolerance(ref, scale, size, d, max(now), BF16, np.abs(V).max()), "out")
        close_lse(f64(lse), rl, size, d + 8)


def test_binding_refusals(sfi):
    c = Cache(sfi, 4, 2, 64, I8, 16, [20])
    q, out = normal((1, 4, 64), BF16, 80), torch.empty(1, 4, 64, device="cuda")
    ws = sfi.paged_workspace(c.lay)
    plain = sfi.PagedLayout(4, 2, 64, BF16, 16, c.n_pages, c.table, c.len)
    with pytest.raises(ValueError):
        sfi.sfi_paged_attn_q8(plain, q, c.k, c.v, out, None, ws)
    with pytest.raises(ValueError):
        sfi.sfi_paged_attn(c.lay, q, c.k, c.v, out, None, ws)
    for bad in (dict(q=q.half()), dict(q=q[:, :2]), dict(k=c.k[:, :-16]), dict(k=c.k.view(torch.int8)), dict(out=out.bfloat16())):
        args = dict(q=q, k=c.k, v=c.v, out=out, ws=ws)
        args.update(bad)
        with pytest.raises(ValueError):
            sfi.sfi_paged_attn_q8(c.lay, **args)
    new = normal((1, 2, 64), BF16, 81)
    with pytest.raises(ValueError):
        sfi.sfi_paged_append_q8(c.lay, new, new.float(), c.k, c.v, None, ws)
    with pytest.raises(ValueError):
        sfi.sfi_paged_append_q8(c.lay, new.half(), new.half(), c.k, c.v, None, ws)
