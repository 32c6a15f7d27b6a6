"""Norm and rotation of query and key heads (sfi_qk_norm_rope) against the 64-bit restatement."""
import numpy as np
import pytest
import torch

import oracle.heads_oracle as H
from tests.paged_testlib import close, f64, ints, normal
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def tolerance(ref, size, dtype):
    """Elementwise bound.  fp32 inside: the sum of squares is off by 13 roundings (8 products and sums
    in a lane, 4 between lanes, the mean's), which the root halves; rsqrt by 2^-22, two products
    by 2^-24 each: below 2^-20 of a normed element.  Cosine and sine are off by 2 last places
    (2^-23), and by 2 pi (2^-26 for the angle's rounding to fp32 + 2^-32 for its 32 bits)
    < 2^-23; the rotation's products and sum by 3 * 2^-24.  In all below 2^-19 of the
    magnitudes that are added.  Then half a step of the output's type."""
    off = size * 2.0 ** -19
    return off + torch.finfo(dtype).eps / 2 * (np.abs(ref) + off) + 2.0 ** -140


def run(sfi, hq, hkv, d, dtype, pos, rot=None, theta=10000.0, interleaved=False, eps=1e-6, weights=True, offset=0, seed=1,
        joint=False, in_place=False, scale=1.0, inv_freq=None):
    rows = len(pos)
    if joint:  # slices of one projection, and of one buffer for the outputs
        x = normal((rows, hq + 2 * hkv, d), dtype, seed) * scale
        q, k = x[:, :hq], x[:, hq:hq + hkv]
    else:
        q, k = normal((rows, hq, d), dtype, seed) * scale, normal((rows, hkv, d), dtype, seed + 1) * scale
    wq, wk = ((1 + 0.3 * normal((d,), F32, seed + i)).to(dtype) if weights and eps is not None else None for i in (2, 3))
    before = [f64(t) for t in (q, k)]
    lay = sfi.RotaryLayout(hq, hkv, d, dtype, ints(pos), rotary_dim=rot, theta=theta, interleaved=interleaved, eps=eps,
                           pos_offset=offset, inv_freq=inv_freq)
    qo, ko = (q, k) if in_place else (torch.full_like(q.contiguous(), 7.0), torch.full_like(k.contiguous(), 7.0))
    sfi.sfi_qk_norm_rope(lay, q if hq else None, k if hkv else None, qo if hq else None, ko if hkv else None,
                         wq if hq else None, wk if hkv else None)
    torch.cuda.synchronize()
    r = d if rot is None else rot
    freq = inv_freq if inv_freq is not None else [theta ** (-2.0 * i / r) for i in range(r // 2)]
    for got, x, w, name in ((qo, before[0], wq, "q"), (ko, before[1], wk, "k")):
        if got.numel() == 0:
            continue
        ref, size = H.norm_rope(x, None if w is None else f64(w), [p + offset for p in pos], freq, interleaved, eps)
        close(f64(got), ref, tolerance(ref, size, dtype), name)
        if not in_place:
            again = f64(x_) if (x_ := {"q": q, "k": k}[name]) is not None else None
            assert np.array_equal(again, x), "an input changed"
    return qo, ko


@pytest.mark.parametrize("hq,hkv,d,dtype,rot,interleaved", [
    (8, 2, 128, BF16, None, False), (8, 2, 64, BF16, None, False), (4, 4, 128, F32, None, False), (3, 1, 64, F32, None, False),
    (8, 2, 128, BF16, None, True), (5, 1, 64, F32, None, True), (8, 2, 128, BF16, 64, False), (8, 2, 128, F32, 32, True),
    (2, 1, 64, BF16, 8, False), (2, 1, 64, BF16, 8, True), (7, 3, 128, F32, 40, False), (1, 1, 128, BF16, 120, False),
    (16, 1, 64, BF16, 24, True), (33, 11, 64, F32, 16, False), (9, 3, 128, BF16, 0, False),
])
def test_matches_restatement(sfi, hq, hkv, d, dtype, rot, interleaved):
    run(sfi, hq, hkv, d, dtype, [0, 1, 5, 1000, 77], rot, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(sfi, dtype, interleaved):
    """Positions whose angle in fp32 would be off by radians; offsets on both sides of zero."""
    run(sfi, 2, 1, 64, dtype, [131072, 4000003, (1 << 30) + 7, (1 << 31) - 1, -1, -(1 << 31)], interleaved=interleaved)
    run(sfi, 2, 1, 64, dtype, [1, 0, 300, -5], offset=-1, interleaved=interleaved)
    run(sfi, 2, 1, 64, dtype, [(1 << 31) - 1, 3], offset=(1 << 31) - 1, interleaved=interleaved)


def test_other_frequencies(sfi):
    run(sfi, 4, 2, 128, F32, [0, 9, 12345], theta=500000.0)
    freq = [0.0, 1e-9, -0.5, 2.0, 6.5, 100.25, 0.125, 3.0]  # none, tiny, backwards, more than a turn a position
    for il in (False, True):
        run(sfi, 4, 2, 64, F32, [0, 1, 9, 12345], rot=16, inv_freq=freq, interleaved=il)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_variants(sfi, dtype):
    pos = [4, 0, 12]
    run(sfi, 4, 1, 128, dtype, pos, eps=None)                    # rotation alone
    run(sfi, 4, 1, 128, dtype, pos, weights=False)
    run(sfi, 4, 1, 64, dtype, pos, rot=0)                        # norm alone
    run(sfi, 4, 1, 64, dtype, pos, eps=0.0, scale=1e-12)
    run(sfi, 4, 1, 64, dtype, pos, eps=1.0, scale=1e-12)
    run(sfi, 4, 1, 64, dtype, pos, scale=1e15)
    run(sfi, 4, 0, 64, dtype, pos)
    run(sfi, 0, 3, 128, dtype, pos)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_joint_projection(sfi, dtype, in_place):
    run(sfi, 6, 2, 128, dtype, list(range(90, 130)), joint=True, in_place=in_place)
    run(sfi, 3, 1, 64, dtype, [5], joint=True, in_place=in_place)


def test_row_of_zeros_and_what_is_not_finite(sfi):
    q = normal((4, 2, 64), F32, 3)
    q[0], q[1, 0, 5], q[2, 1, 60] = 0, float("inf"), float("nan")
    k = normal((4, 1, 64), F32, 4)
    lay = sfi.RotaryLayout(2, 1, 64, F32, ints([3, 3, 3, 3]), rotary_dim=32, eps=1e-6)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    sfi.sfi_qk_norm_rope(lay, q, k, qo, ko)
    assert (qo[0] == 0).all() and torch.isfinite(qo[3]).all() and torch.isfinite(ko).all()
    assert qo[1, 0].isnan().any() and torch.isfinite(qo[1, 1]).all()
    assert qo[2, 1].isnan().all() and torch.isfinite(qo[2, 0]).all()
    # without a norm only the pair is touched
    lay = sfi.RotaryLayout(2, 1, 64, F32, ints([3, 3, 3, 3]), rotary_dim=32, eps=None)
    sfi.sfi_qk_norm_rope(lay, q, k, qo, ko)
    bad = ~torch.isfinite(qo)
    assert bad[1, 0].nonzero().flatten().tolist() == [5, 21] and bad[2, 1].nonzero().flatten().tolist() == [60]
    assert int(bad.sum()) == 3 and (qo[0] == 0).all()


@pytest.mark.parametrize("rows,hq,hkv", [(1, 32, 8), (64, 32, 8), (700, 32, 8), (2500, 3, 1), (20000, 1, 1)])
def test_rows_over_warps(sfi, rows, hq, hkv):
    """A row's heads over several warps, or a warp a row: each row alone gives the same bits."""
    d = 128
    q, k = normal((rows, hq, d), BF16, 5), normal((rows, hkv, d), BF16, 6)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 3
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    sfi.sfi_qk_norm_rope(sfi.RotaryLayout(hq, hkv, d, BF16, pos), q, k, qo, ko)
    for t in sorted({0, rows // 2, rows - 1}):
        q1, k1 = torch.empty_like(q[:1]), torch.empty_like(k[:1])
        sfi.sfi_qk_norm_rope(sfi.RotaryLayout(hq, hkv, d, BF16, pos[t:t + 1]), q[t:t + 1], k[t:t + 1], q1, k1)
        assert torch.equal(q1[0], qo[t]) and torch.equal(k1[0], ko[t])


def test_stream_and_graph(sfi):
    """On a stream of the caller's, and captured: a replay reads the positions of its time."""
    q, k = normal((5, 4, 64), BF16, 7), normal((5, 2, 64), BF16, 8)
    pos = ints([1, 2, 3, 4, 5])
    lay = sfi.RotaryLayout(4, 2, 64, BF16, pos, pos_offset=-1)
    qo, ko, q2, k2 = (torch.empty_like(t) for t in (q, k, q, k))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sfi.sfi_qk_norm_rope(lay, q, k, qo, ko, stream=st)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sfi.sfi_qk_norm_rope(lay, q, k, q2, k2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    pos += 100
    graph.replay()
    sfi.sfi_qk_norm_rope(lay, q, k, qo, ko)
    torch.cuda.synchronize()
    assert torch.equal(qo, q2) and torch.equal(ko, k2) and not torch.equal(qo, q)


def test_empty(sfi):
    e = torch.empty(0, 2, 64, device="cuda")
    sfi.sfi_qk_norm_rope(sfi.RotaryLayout(2, 2, 64, F32, ints([])), e, e, e, e)


def test_binding_refusals(sfi):
    q, k = normal((4, 2, 64), F32, 1), normal((4, 1, 64), F32, 2)
    lay = sfi.RotaryLayout(2, 1, 64, F32, ints([0, 1, 2, 3]))
    for bad in (dict(q=q.bfloat16()), dict(q=q[:3]), dict(q=q.cpu()), dict(k=k.expand(4, 2, 64)), dict(q_weight=torch.ones(32, device="cuda")),
                dict(k_weight=torch.ones(64, device="cuda").bfloat16()), dict(q=None), dict(q=q[:1].expand(4, 2, 64)), dict(q=q[..., ::2])):
        args = dict(q=q, k=k, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        args.update(bad)
        with pytest.raises(ValueError):
            sfi.sfi_qk_norm_rope(lay, **args)
    with pytest.raises(ValueError):
        sfi.RotaryLayout(2, 1, 64, F32, ints([0]), inv_freq=[1.0])
    with pytest.raises(ValueError):
        sfi.RotaryLayout(2, 1, 64, F32, None)
    with pytest.raises(ValueError):
        sfi.RotaryLayout(2, 1, 64, F32, ints([0]), pos_offset=1 << 31)
