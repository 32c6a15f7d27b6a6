"""Prompt attention (sfi_prefill_attn) against the fp64 restatement: packed
sequences of one token to several key blocks, chunks after earlier context,
rows that see nothing, every group size, strided rows, and what lies outside
the sequences."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import bf16_tolerance, close, close_lse, f64, ints, normal, offsets
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def run(sfi, q, k, v, cu_q, cu_k, ws=None):
    lay = sfi.PackedLayout(q.shape[1], k.shape[1], q.shape[2], BF16, ints(cu_q), ints(cu_k), q.shape[0], k.shape[0])
    ws = sfi.prefill_workspace(lay) if ws is None else ws
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sfi.sfi_prefill_attn(lay, q, k, v, out, lse, ws)
    torch.cuda.synchronize()
    assert sfi.sfi_read_status(ws) == 0
    return out, lse


def check(q, k, v, cu_q, cu_k, out, lse, rows=None):
    ref, rl, scale, size = P.prefill(f64(q), f64(k), f64(v), cu_q, cu_k, rows)
    inside = ~np.isnan(rl)
    assert not (cu_q[-1] > cu_q[0]) or inside.any()
    d = q.shape[2]
    close(f64(out)[inside], ref[inside], bf16_tolerance(ref, scale, size, d)[inside], "out")
    close_lse(f64(lse)[inside], rl[inside], size[inside], d)
    if rows is not None:
        return
    # rows of no sequence stay as they were
    assert (f64(out)[~inside] == 7.0).all() and (f64(lse)[~inside] == 7.0).all()


CASES = [
    # (H_q, H_kv, d, query lengths, key lengths or None)
    (8, 2, 128, [1], None),
    (8, 2, 64, [1, 1, 1], None),
    (8, 2, 128, [129, 1, 64, 300], None),
    (4, 1, 64, [128, 127, 31, 33, 0, 260], None),
    (2, 2, 128, [256, 257, 255], None),
    (3, 1, 128, [200, 43, 5], None),      # 128 % G != 0: 42 tokens a tile
    (10, 2, 64, [90, 26], None),
    (7, 1, 128, [150], None),
    (16, 1, 128, [40, 9], None),
    (8, 1, 64, [500], None),
    (8, 2, 128, [5, 70], [300, 70]),      # chunks after earlier context
    (4, 2, 64, [130, 1, 17], [641, 129, 128]),
    (8, 2, 128, [60, 4, 0, 3], [20, 0, 9, 3]),  # rows without keys, and a sequence without queries
    (2, 1, 64, [300], [70]),              # a whole tile without keys
]


@pytest.mark.parametrize("hq,hkv,d,nq,nk", CASES)
def test_prefill_matches_oracle(sfi, hq, hkv, d, nq, nk):
    cu_q, cu_k = offsets(nq), offsets(nk or nq)
    q = normal((cu_q[-1], hq, d), BF16, 1)
    k = normal((cu_k[-1], hkv, d), BF16, 2)
    v = normal((cu_k[-1], hkv, d), BF16, 3)
    out, lse = run(sfi, q, k, v, cu_q, cu_k)
    check(q, k, v, cu_q, cu_k, out, lse)
    again, lse2 = run(sfi, q, k, v, cu_q, cu_k)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


CUT = [
    # few tiles over many keys, so that they are cut along the keys and joined
    (8, 2, 128, [70, 64, 5], [2000, 1500, 3001]),
    (8, 2, 64, [33, 1], [1025, 4000]),
    (3, 1, 128, [50], [1700]),
    (16, 1, 64, [20, 9], [900, 2222]),
    (4, 1, 128, [1030], None),                      # a whole prompt: some parts see no key of some rows
    (4, 1, 64, [200, 3, 0, 300], [90, 3, 500, 1111]),  # rows without keys among them
]


@pytest.mark.parametrize("hq,hkv,d,nq,nk", CUT)
def test_cut_tiles_are_joined(sfi, hq, hkv, d, nq, nk):
    cu_q, cu_k = offsets(nq), offsets(nk or nq)
    assert cu_k[-1] >= 1024
    q = normal((cu_q[-1] + 2, hq, d), BF16, 1)
    k, v = normal((cu_k[-1] + 3, hkv, d), BF16, 2), normal((cu_k[-1] + 3, hkv, d), BF16, 3)
    k[cu_k[-1]:], v[cu_k[-1]:] = float("nan"), float("nan")
    out, lse = run(sfi, q, k, v, cu_q, cu_k)
    rows = set(range(0, cu_q[-1], 1 if cu_q[-1] < 200 else 13)) | {x for y in cu_q for x in (y - 1, y)}
    check(q, k, v, cu_q, cu_k, out, lse, rows)
    assert (out[cu_q[-1]:] == 7.0).all() and (lse[cu_q[-1]:] == 7.0).all()
    again, lse2 = run(sfi, q, k, v, cu_q, cu_k)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_last_wave_is_cut(sfi):
    """More tiles of one length than SMs: the last, partly filled wave's are cut (8 KV heads x 25
    tiles of 64 tokens, 48 of the 200 on a GPU with 152 SMs), the others are not."""
    hq, hkv, d, nq, nk = 32, 8, 64, 1600, 3400
    q, k, v = normal((nq, hq, d), BF16, 1), normal((nk, hkv, d), BF16, 2), normal((nk, hkv, d), BF16, 3)
    out, lse = run(sfi, q, k, v, [0, nq], [0, nk])
    check(q, k, v, [0, nq], [0, nk], out, lse, set(range(0, nq, 67)) | {0, 63, 64, nq - 1})
    # the tiles of a call with one head group are all cut: the same within the rounding of both
    one, lse1 = run(sfi, q[:, :4].contiguous(), k[:, :1].contiguous(), v[:, :1].contiguous(), [0, nq], [0, nk])
    check(q[:, :4], k[:, :1], v[:, :1], [0, nq], [0, nk], one, lse1, set(range(0, nq, 31)))


def test_growing_scores_rescale(sfi):
    """Keys whose scores climb by far more than the lazy rescaling allows, block after block, and
    then fall: every row's maximum moves several times."""
    n, d = 700, 128
    q = normal((n, 4, d), BF16, 1)
    k = normal((n, 1, d), BF16, 2)
    ramp = torch.linspace(0.1, 6.0, n, device="cuda") * (1 + (torch.arange(n, device="cuda") % 131 == 7))
    k = (k.float() * ramp[:, None, None]).to(BF16)
    v = normal((n, 1, d), BF16, 3)
    out, lse = run(sfi, q, k, v, [0, n], [0, n])
    check(q, k, v, [0, n], [0, n], out, lse)


def test_rows_outside_the_sequences(sfi):
    """Slots before the first and behind the last sequence stay untouched, and NaN or infinities
    there and in the neighbours' rows reach nobody."""
    hq, hkv, d = 8, 2, 128
    cu_q, cu_k = [5, 75, 76, 236], [3, 73, 203, 363]
    q = normal((300, hq, d), BF16, 1)
    k = normal((400, hkv, d), BF16, 2)
    v = normal((400, hkv, d), BF16, 3)
    for t, cu in ((k, cu_k), (v, cu_k)):
        t[:cu[0]] = float("nan")
        t[cu[-1]:] = float("inf")
    out, lse = run(sfi, q, k, v, cu_q, cu_k)
    check(q, k, v, cu_q, cu_k, out, lse)
    # the middle sequence's rows spoilt: the others keep their bits
    v2, k2 = v.clone(), k.clone()
    v2[cu_k[1]:cu_k[2]] = float("nan")
    k2[cu_k[1]:cu_k[2]] = float("-inf")
    out2, lse2 = run(sfi, q, k2, v2, cu_q, cu_k)
    for a, b in ((0, 1), (2, 3)):
        assert torch.equal(out[cu_q[a]:cu_q[b]], out2[cu_q[a]:cu_q[b]])
        assert torch.equal(lse[cu_q[a]:cu_q[b]], lse2[cu_q[a]:cu_q[b]])
    # a NaN key reaches only the rows that attend to it
    k3 = k.clone()
    k3[cu_k[2] + 100] = float("nan")
    out3, _ = run(sfi, q, k3, v, cu_q, cu_k)
    assert torch.equal(out[cu_q[2]:cu_q[2] + 100], out3[cu_q[2]:cu_q[2] + 100])
    assert torch.isnan(out3[cu_q[2] + 100:cu_q[3]]).all()


def test_strided_rows(sfi):
    """q, k and v as slices of one projection, out as a slice of a wider buffer."""
    hq, hkv, d, n = 8, 2, 64, 210
    both = normal((n, (hq + 2 * hkv) * d + 8), BF16, 4)
    q = both[:, :hq * d].view(n, hq, d)
    k = both[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    v = both[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(n, hkv, d)
    wide = torch.full((n, hq * d + 16), 5.0, dtype=BF16, device="cuda")
    out, lse = wide[:, 8:8 + hq * d].view(n, hq, d), torch.empty(n, hq, device="cuda")
    lay = sfi.PackedLayout(hq, hkv, d, BF16, ints([0, 100, n]), ints([0, 100, n]), n, n)
    ws = sfi.prefill_workspace(lay)
    sfi.sfi_prefill_attn(lay, q, k, v, out, lse, ws)
    check(q, k, v, [0, 100, n], [0, 100, n], out, lse)
    assert (wide[:, :8] == 5.0).all() and (wide[:, 8 + hq * d:] == 5.0).all()
    same, _ = run(sfi, q.contiguous(), k.contiguous(), v.contiguous(), [0, 100, n], [0, 100, n])
    assert torch.equal(same, out)
    sfi.sfi_prefill_attn(lay, q, k, v, out, None, ws)  # without lse
    assert torch.equal(same, out) and sfi.sfi_read_status(ws) == 0


def test_bad_offsets_are_flagged(sfi):
    """Descending or overlong offsets: the status names them, the other sequences are computed."""
    q, k, v = normal((96, 4, 64), BF16, 1), normal((96, 1, 64), BF16, 2), normal((96, 1, 64), BF16, 3)
    good, _ = run(sfi, q, k, v, [0, 40, 96], [0, 40, 96])
    for cu in ([0, 40, 97], [0, 40, 39], [-1, 40, 96]):
        lay = sfi.PackedLayout(4, 1, 64, BF16, ints(cu), ints(cu), 96, 96)
        ws = sfi.prefill_workspace(lay)
        out = torch.full_like(q, 7.0)
        sfi.sfi_prefill_attn(lay, q, k, v, out, None, ws)
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == sfi.SFI_DEV_LEN_OVER_CAP
        want = torch.full_like(q, 7.0)
        if cu[0] == 0:
            want[:40] = good[:40]
        else:
            want[40:] = good[40:]
        assert torch.equal(out, want)


def test_many_short_sequences(sfi):
    """More sequences than a warp scans at once, of every length from 0 to 9 tokens."""
    lens = [(7 * i) % 10 for i in range(100)]
    cu = offsets(lens)
    q, k, v = normal((cu[-1], 4, 64), BF16, 1), normal((cu[-1], 2, 64), BF16, 2), normal((cu[-1], 2, 64), BF16, 3)
    out, lse = run(sfi, q, k, v, cu, cu)
    check(q, k, v, cu, cu, out, lse)


def test_no_queries_and_no_keys(sfi):
    lay = sfi.PackedLayout(4, 2, 64, BF16, ints([0, 0]), ints([0, 3]), 0, 3)
    ws = sfi.prefill_workspace(lay)
    e = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    kv = normal((3, 2, 64), BF16, 1)
    sfi.sfi_prefill_attn(lay, e, kv, kv, e, None, ws)
    q, none = normal((5, 4, 64), BF16, 1), torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    out, lse = run(sfi, q, none, none, [0, 5], [0, 0])
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_captured_and_other_stream(sfi):
    """Two captured calls that share a workspace, replayed on new inputs on a side stream."""
    cu = [0, 100, 333]
    q, k, v = normal((333, 8, 128), BF16, 1), normal((333, 2, 128), BF16, 2), normal((333, 2, 128), BF16, 3)
    lay = sfi.PackedLayout(8, 2, 128, BF16, ints(cu), ints(cu), 333, 333)
    ws = sfi.prefill_workspace(lay)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sfi.sfi_prefill_attn(lay, q, k, v, out, None, ws)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            sfi.sfi_prefill_attn(lay, q, k, v, out, None, ws)
            sfi.sfi_prefill_attn(lay, out, k, v, out2, None, ws)
        q.copy_(normal(q.shape, BF16, 9))
        g.replay()
        st.synchronize()
    one, _ = run(sfi, q, k, v, cu, cu)
    two, _ = run(sfi, one, k, v, cu, cu)
    assert torch.equal(out, one) and torch.equal(out2, two)


def test_wait_limit(sfi):
    """A one-clock limit: waits give up, the status says so, the call returns; afterwards the
    default limit gives the bytes from before."""
    n = 1500
    q, k, v = normal((n, 8, 128), BF16, 1), normal((n, 2, 128), BF16, 2), normal((n, 2, 128), BF16, 3)
    good, _ = run(sfi, q, k, v, [0, n], [0, n])
    lay = sfi.PackedLayout(8, 2, 128, BF16, ints([0, n]), ints([0, n]), n, n)
    ws = sfi.prefill_workspace(lay)
    out = torch.empty_like(q)
    sfi.lib.sfi_set_wait_limit(1)
    try:
        for _ in range(2):
            sfi.sfi_prefill_attn(lay, q, k, v, out, None, ws)
            assert sfi.sfi_read_status(ws) == sfi.SFI_DEV_WAIT_TIMEOUT
    finally:
        sfi.lib.sfi_set_wait_limit(0)
    ws.zero_()
    again, _ = run(sfi, q, k, v, [0, n], [0, n], ws)
    assert torch.equal(good, again)


def test_expanded_rows_are_refused(sfi):
    q, k = (torch.zeros(9, h, 64, device="cuda", dtype=BF16) for h in (4, 2))
    lay = sfi.PackedLayout(4, 2, 64, BF16, ints([0, 9]), ints([0, 9]), 9, 9)
    ws, out = sfi.prefill_workspace(lay), torch.empty_like(q)
    for a in ((q[:1].expand(9, 4, 64), k, k, out), (q, k[:1].expand(9, 2, 64), k, out),
              (q, k, k[:1].expand(9, 2, 64), out), (q, k, k, out[:1].expand(9, 4, 64))):
        with pytest.raises(ValueError):
            sfi.sfi_prefill_attn(lay, *a, None, ws)


@pytest.mark.parametrize("hq,hkv", [(128, 8), (100, 10)])  # output by boxes, and by rows
def test_offsets_past_32_bits(sfi, hq, hkv):
    """A short sequence behind more than 2^31 elements of q and out, and of k and v by their strides."""
    d, first, n = 128, (1 << 31) // (hq * 128) + 100, 150
    cu, ck = [first, first + n], [70000, 70000 + n]
    q = torch.empty(first + n + 3, hq, d, dtype=BF16, device="cuda")
    wide = torch.empty(70000 + n, 40000, dtype=BF16, device="cuda")
    k, v = (wide[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    qs, ks, vs = normal((n, hq, d), BF16, 1), normal((n, hkv, d), BF16, 2), normal((n, hkv, d), BF16, 3)
    q[first:first + n], k[70000:], v[70000:] = qs, ks, vs
    lay = sfi.PackedLayout(hq, hkv, d, BF16, ints(cu), ints(ck), q.shape[0], k.shape[0])
    ws, out = sfi.prefill_workspace(lay), torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    sfi.sfi_prefill_attn(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    rows = np.array([0, 1, 63, 64, 127, 128, n - 1])
    ref, rl, scale, size = P.prefill(f64(qs), f64(ks), f64(vs), [0, n], [0, n], set(rows.tolist()))
    close(f64(out[first:first + n])[rows], ref[rows], bf16_tolerance(ref, scale, size, d)[rows], "out")
    close_lse(f64(lse[first:first + n])[rows], rl[rows], size[rows], d)
    assert bool((out[:first] == 7).all()) and bool((out[first + n:] == 7).all())
