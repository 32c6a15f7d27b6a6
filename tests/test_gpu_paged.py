"""Attention over a paged cache (sfi_paged_attn) against the fp64 restatement: both types, page
sizes that end inside a tile, lengths from 0, every group size, far pages, garbage in unused rows."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import close, close_lse, f32_tolerance, f64, ints, normal, pool_of
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


class Cache:
    def __init__(self, hq, hkv, d, dtype, page, lens, seed=1):
        self.hq, self.hkv, self.d, self.dtype, self.page = hq, hkv, d, dtype, page
        self.lens = list(lens)
        self.n_pages, self.rows = pool_of(lens, page, 3, seed)
        self.table, self.len = ints(self.rows.tolist()), ints(self.lens)
        self.q = normal((len(lens), hq, d), dtype, seed + 1)
        self.k = normal((self.n_pages, hkv, page, d), dtype, seed + 2)
        self.v = normal((self.n_pages, hkv, page, d), dtype, seed + 3)

    def layout(self, sfi, **kw):
        return sfi.PagedLayout(self.hq, self.hkv, self.d, self.dtype, self.page, self.n_pages, self.table, self.len, **kw)

    def run(self, sfi, ws=None, status=0, k=None, v=None, **kw):
        lay = self.layout(sfi, **kw)
        ws = sfi.paged_workspace(lay) if ws is None else ws
        out = torch.full((len(self.lens), self.hq, self.d), 7.0, device="cuda")
        lse = torch.full((len(self.lens), self.hq), 7.0, device="cuda")
        sfi.sfi_paged_attn(lay, self.q, self.k if k is None else k, self.v if v is None else v, out, lse, ws)
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == status
        return out, lse

    def check(self, out, lse):
        ref, rl, scale, size = P.paged(f64(self.q), f64(self.k), f64(self.v), self.rows, self.lens)
        tol = f32_tolerance(ref, scale, size, self.d, max(self.lens), self.dtype == BF16)
        close(f64(out), ref, tol, "out")
        close_lse(f64(lse), rl, size, self.d)


CASES = [
    # (H_q, H_kv, d, dtype, page size, lengths)
    (8, 2, 128, BF16, 16, [1]),
    (8, 2, 128, BF16, 16, [0, 15, 16, 17, 0, 300]),
    (8, 2, 64, BF16, 32, [700, 33, 64]),
    (4, 4, 128, BF16, 48, [500, 47, 49]),
    (8, 1, 128, BF16, 64, [2100]),
    (16, 1, 128, BF16, 16, [130, 1]),
    (10, 1, 64, BF16, 256, [800, 255]),
    (3, 1, 128, BF16, 16, [77]),
    (14, 2, 128, BF16, 1, [40, 7]),        # pages gathered row by row
    (8, 2, 128, BF16, 5, [203, 4, 0]),
    (6, 2, 64, BF16, 24, [100, 24, 25]),
    (16, 1, 64, BF16, 20, [333]),
    (8, 2, 128, F32, 16, [0, 15, 16, 17, 300]),
    (8, 2, 64, F32, 20, [700, 33, 1]),
    (2, 2, 128, F32, 1, [50, 3]),
    (7, 1, 64, F32, 3, [101]),
    (16, 1, 128, F32, 64, [200, 64]),
    (5, 1, 128, F32, 8, [99, 8]),
    (12, 1, 64, F32, 48, [300]),
]


@pytest.mark.parametrize("hq,hkv,d,dtype,page,lens", CASES)
def test_paged_matches_oracle(sfi, hq, hkv, d, dtype, page, lens):
    c = Cache(hq, hkv, d, dtype, page, lens)
    out, lse = c.run(sfi)
    c.check(out, lse)
    again, lse2 = c.run(sfi)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,page", [(BF16, 16), (BF16, 24), (F32, 20)])
def test_unused_rows_may_hold_anything(sfi, dtype, page):
    """NaN behind every sequence's end and in every page that nobody holds; table entries behind
    the held ones point nowhere."""
    c = Cache(8, 2, 128, dtype, page, [100, 0, 37, page, 1])
    good, _ = c.run(sfi)
    c.check(*c.run(sfi))
    used = torch.zeros(c.n_pages, page, dtype=torch.bool)
    for b, n in enumerate(c.lens):
        for i in range(n):
            used[c.rows[b, i // page], i % page] = True
    for pool in (c.k, c.v):
        pool.masked_fill_(~used.cuda()[:, None, :, None], float("nan"))
    c.table[c.table < 0] = 1 << 30
    out, _ = c.run(sfi)
    assert torch.equal(out, good)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_scores_rescale(sfi, dtype):
    c = Cache(4, 1, 128, dtype, 16, [1500])
    ramp = torch.linspace(0.1, 6.0, 1600, device="cuda")[:1500]
    for i in range(94):
        part = ramp[i * 16:(i + 1) * 16]
        c.k[c.rows[0, i], :, :len(part)] *= part[None, :, None].to(dtype)
    c.check(*c.run(sfi))


def test_many_sequences(sfi):
    """More sequences than CTAs, with idle slots between: pieces of many units in one CTA."""
    c = Cache(4, 2, 64, BF16, 16, [(i * 7) % 41 for i in range(300)])
    c.check(*c.run(sfi))


def test_largest_batch(sfi):
    c = Cache(4, 4, 64, BF16, 16, [1 + (i % 3) for i in range(1024)])
    c.check(*c.run(sfi))


@pytest.mark.parametrize("hq,hkv,d,dtype,page,lens", [
    (4, 2, 64, BF16, 16, [70000, 8191, 0, 130001]),  # units of far more than 16 pieces
    (32, 8, 64, BF16, 20, [24001] * 4),              # several units a share, gathered rows
    (8, 8, 128, BF16, 64, [24576] * 12),             # the same by boxes, one head a group
    (2, 2, 64, F32, 16, [90000, 40003, 90001]),
    (8, 2, 128, BF16, 16, [200000, 160001, 0, 280000]),  # large shares, units of up to 34
    (8, 8, 128, BF16, 32, [16390] * 10),                 # and of a few pieces
])
def test_long_units_are_cut_and_joined(sfi, hq, hkv, d, dtype, page, lens):
    """Lengths at which units are cut into many pieces, and shares hold several units: the first,
    a middle and the last sequence, and the first and last KV head of each."""
    c = Cache(hq, hkv, d, dtype, page, lens, seed=60)
    out, lse = c.run(sfi)
    again, lse2 = c.run(sfi)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    G = hq // hkv
    for b in sorted({0, len(lens) // 2, len(lens) - 1}):
        ids = c.rows[b][:-(-lens[b] // page)].tolist()
        for g in sorted({0, hkv - 1}):
            rows = torch.tensor(ids, device="cuda", dtype=torch.long)
            K, V = (f64(x[rows, g].reshape(-1, d)) for x in (c.k, c.v))
            for h in (g * G, g * G + G - 1):
                ref, rl, scale, size = (np.asarray(x)[None] for x in P.attend(f64(c.q[b, h]), K, V, lens[b]))
                tol = f32_tolerance(ref, scale, size, d, lens[b], dtype == BF16)
                close(f64(out[b, h])[None], ref, tol, ("out", b, h))
                close_lse(f64(lse[b, h])[None], rl, size, d, ("lse", b, h))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_apart(sfi, dtype):
    """K and V of a page side by side in one allocation."""
    c = Cache(8, 2, 64, dtype, 16, [90, 200])
    good, _ = c.run(sfi)
    both = torch.stack([c.k, c.v], 1).contiguous()
    out, _ = c.run(sfi, k=both[:, 0], v=both[:, 1], page_stride=both.stride(0))
    assert torch.equal(out, good)


@pytest.mark.parametrize("dtype,page", [(BF16, 16), (BF16, 20), (F32, 16)])
def test_offsets_past_32_bits(sfi, dtype, page):
    """Pages so far apart that element and byte offsets need more than 32 bits."""
    c = Cache(4, 1, 64, dtype, page, [page * 2 + 3])
    good, _ = c.run(sfi)
    stride = (1 << 30) + 64
    rooms = []
    for pool in (c.k, c.v):
        far = torch.empty((c.n_pages - 1) * stride + page * 64, dtype=dtype, device="cuda")
        view = far.as_strided(tuple(pool.shape), (stride, page * 64, 64, 1))
        view.copy_(pool)
        rooms.append(view)
    out, _ = c.run(sfi, k=rooms[0], v=rooms[1], page_stride=stride)
    assert torch.equal(out, good)


def test_agrees_with_the_contiguous_cache(sfi):
    """The same rows in pages and in one slab per sequence (sfi_slow_attn)."""
    lens = [400, 33]
    c = Cache(8, 2, 128, BF16, 16, lens)
    out, _ = c.run(sfi)
    cap = 416
    k, v = (torch.zeros(2, 2, cap, 128, dtype=BF16, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        for i in range(-(-n // 16)):
            k[b, :, i * 16:(i + 1) * 16] = c.k[c.rows[b, i]]
            v[b, :, i * 16:(i + 1) * 16] = c.v[c.rows[b, i]]
    lay = sfi.Layout(8, 2, 128, BF16, [0, 2 * cap * 128], [cap, cap], lens, cap)
    dense = torch.empty_like(out)
    sfi.sfi_slow_attn(lay, c.q, k, v, dense, None, None, sfi.alloc_workspace(lay))
    assert float((dense - out).abs().max()) <= 1e-2  # the contiguous call's own bound


def test_bad_lengths_and_pages_are_flagged(sfi):
    for dtype, page in ((BF16, 16), (BF16, 20), (F32, 16)):
        c = Cache(8, 2, 64, dtype, page, [90, 50])
        good, _ = c.run(sfi)
        c.len.copy_(ints([90, -5]))
        out, lse = c.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP)
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        # (the other's rows are split elsewhere now, and summed in another order)
        ref, _, scale, size = P.paged(f64(c.q), f64(c.k), f64(c.v), c.rows, c.lens)
        close(f64(out)[0], ref[0], f32_tolerance(ref, scale, size, 64, 90, dtype == BF16)[0], "out")
        c.len.copy_(ints([90, 50]))
        c.table[1, 1] = c.n_pages
        out, _ = c.run(sfi, status=sfi.SFI_DEV_BAD_INDEX)
        assert torch.equal(out[0], good[0])
        c.table[1, 1] = -7
        out2, _ = c.run(sfi, status=sfi.SFI_DEV_BAD_INDEX)
        assert torch.equal(out2, out)  # page 0 both times
        # longer than the table's row: taken as full, its unheld entries are bad pages
        c.len.copy_(ints([1 << 30, 50]))
        c.table[1, 1] = int(c.rows[1, 1])
        c.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP | sfi.SFI_DEV_BAD_INDEX)


def test_captured_calls_share_a_workspace(sfi):
    """Two captured calls of one geometry, one after the other in one graph and in two, replayed on
    a side stream with new lengths."""
    c = Cache(8, 2, 128, BF16, 16, [900, 40, 0])
    lay = c.layout(sfi)
    ws = sfi.paged_workspace(lay)
    outs = [torch.empty(3, 8, 128, device="cuda") for _ in range(3)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sfi.sfi_paged_attn(lay, c.q, c.k, c.v, outs[0], None, ws)
        st.synchronize()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g1, stream=st):
            sfi.sfi_paged_attn(lay, c.q, c.k, c.v, outs[0], None, ws)
            sfi.sfi_paged_attn(lay, c.q, c.v, c.k, outs[1], None, ws)
        with torch.cuda.graph(g2, stream=st):
            sfi.sfi_paged_attn(lay, c.q, c.k, c.v, outs[2], None, ws)
        c.len.copy_(ints([880, 47, 0]))
        for _ in range(2):
            g1.replay()
            g2.replay()
        st.synchronize()
    c.lens = [880, 47, 0]
    one, lse = c.run(sfi)
    c.check(one, lse)
    assert torch.equal(outs[0], one) and torch.equal(outs[2], one)
    assert torch.equal(outs[1], c.run(sfi, k=c.v, v=c.k)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wait_limit(sfi, dtype):
    """A one-clock limit: the waits give up, the status says so, nothing is left in flight.  The
    cache is larger than L2, so that HBM is slower than the arithmetic and some wait is always
    early (of a few thousand rows in L2, every tile has landed when its warp looks)."""
    c = Cache(8, 2, 128, dtype, 16, [1])
    c.lens = [8192] * 64
    c.n_pages = 64 * 512
    c.table = torch.randperm(c.n_pages, device="cuda").view(64, 512).int()
    c.len = ints(c.lens)
    c.q = normal((64, 8, 128), dtype, 1)
    c.k, c.v = (torch.randn(c.n_pages, 2, 16, 128, device="cuda", dtype=dtype) for _ in range(2))
    lay = c.layout(sfi)
    good, _ = c.run(sfi)
    ws = sfi.paged_workspace(lay)
    out = torch.empty_like(good)
    sfi.lib.sfi_set_wait_limit(1)
    try:
        for _ in range(2):
            sfi.sfi_paged_attn(lay, c.q, c.k, c.v, out, None, ws)
            assert sfi.sfi_read_status(ws) == sfi.SFI_DEV_WAIT_TIMEOUT
    finally:
        sfi.lib.sfi_set_wait_limit(0)
    ws.zero_()
    again, _ = c.run(sfi, ws=ws)
    assert torch.equal(good, again)


def test_binding_refusals(sfi):
    c = Cache(8, 2, 64, BF16, 16, [20, 5])
    lay = c.layout(sfi)
    ws, out = sfi.paged_workspace(lay), torch.empty(2, 8, 64, device="cuda")
    for q, k, o in ((c.q.float(), c.k, out), (c.q[:1], c.k, out), (c.q, c.k[:1], out), (c.q, c.k.float(), out),
                    (c.q, c.k, out.to(BF16)), (c.q, c.k.transpose(1, 2), out), (c.q, c.k, out[:, :, :32]),
                    (c.q, c.k.cpu(), out)):
        with pytest.raises(ValueError):
            sfi.sfi_paged_attn(lay, q, k, c.v, o, None, ws)
    with pytest.raises(ValueError):  # pages apart that the layout does not know of
        sfi.sfi_paged_attn(lay, c.q, torch.stack([c.k, c.v], 1)[:, 0], c.v, out, None, ws)
    with pytest.raises(sfi.SfiError):
        sfi.sfi_paged_attn(lay, c.q, c.k, c.v, out, None, ws[:256])
    with pytest.raises(sfi.SfiError):
        sfi.sfi_paged_attn(lay, c.q, c.k, c.v, out, None, None)
