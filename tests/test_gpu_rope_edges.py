"""Norm and rotation of heads (sfi_qk_norm_rope) whose squares leave fp32 on either side, against the
64-bit restatement."""
import numpy as np
import pytest
import torch

import oracle.heads_oracle as H
from tests.paged_testlib import close, f64, ints, normal
from tests.sfi_testlib import load_sfi
from tests.test_gpu_rope import tolerance

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def call(sfi, q, w=None, rot=None, interleaved=False, eps=0.0, pos=None):
    rows, heads, d = q.shape
    pos = [3 + 1000 * i for i in range(rows)] if pos is None else pos
    lay = sfi.RotaryLayout(heads, 0, d, q.dtype, ints(pos), rotary_dim=rot, interleaved=interleaved, eps=eps)
    out = torch.full_like(q, 7.0)
    sfi.sfi_qk_norm_rope(lay, q, None, out, None, w)
    torch.cuda.synchronize()
    return out


def check(sfi, q, w=None, rot=None, interleaved=False, eps=0.0):
    pos = [3 + 1000 * i for i in range(q.shape[0])]
    out = call(sfi, q, w, rot, interleaved, eps, pos)
    r = q.shape[2] if rot is None else rot
    ref, size = H.norm_rope(f64(q), None if w is None else f64(w), pos, [10000.0 ** (-2.0 * i / r) for i in range(r // 2)], interleaved, eps)
    assert np.isfinite(ref).all() and np.abs(ref).max() < torch.finfo(q.dtype).max
    close(f64(out), ref, tolerance(ref, size, q.dtype), "out")
    return out


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,interleaved", [(128, None, False), (64, None, True), (128, 32, False), (64, 8, True), (128, 0, False)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_squares_beyond_fp32(sfi, dtype, d, rot, interleaved, eps):
    """Elements up to the type's largest: the formula's value, whatever the weights."""
    w = ((1 + 0.3 * normal((d,), F32, 5).abs()) * 1.5).to(dtype)
    for scale in (1e14, 1e16, 1e18, 1e20, 1e25, 1e30, 7e37):
        q = normal((3, 5, d), F32, 1).clamp(-4.5, 4.5).mul(scale).to(dtype)
        check(sfi, q, None, rot, interleaved, eps)
        check(sfi, q, w, rot, interleaved, eps)
    q = torch.full((2, 3, d), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    q[:, 1, ::2] *= -1
    q[:, 2, 1:] = 0
    check(sfi, q, w, rot, interleaved, eps)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,rot,interleaved", [(128, None, False), (64, None, True), (128, 32, False), (64, 8, True), (128, 0, False)])
def test_squares_below_fp32(sfi, dtype, d, rot, interleaved):
    """eps = 0, or one that is as small: heads of tiny elements have the length of any others."""
    w = (1 + 0.3 * normal((d,), F32, 5)).to(dtype)
    for scale in (1e-14, 1e-16, 1e-19, 1e-22, 1e-24, 1e-30, 1e-36):
        q = normal((3, 5, d), F32, 1).mul(scale).to(dtype)
        for eps in (0.0, float(np.float32(scale * scale)), 1e-40, 1e-6):
            eps = float(np.float32(eps))
            check(sfi, q, w, rot, interleaved, eps)
    q = torch.zeros(2, 3, d, device="cuda")
    q[0, 0, d - 1] = q[1, 1, 0] = torch.finfo(F32).tiny  # one element alone; a head of the smallest ones
    q[:, 2] = q[:, 0, :1] + torch.finfo(F32).tiny
    q[0, 1], q[1, 0] = 1e-38, -2e-38
    check(sfi, q.to(dtype), w, rot, interleaved)


def test_subnormal_elements(sfi):
    q = torch.randint(-9, 10, (3, 4, 64), generator=torch.Generator().manual_seed(1)).double().mul(2.0 ** -149).float().cuda()
    q[0, 0] = 0
    q[0, 0, 7] = 2.0 ** -149
    check(sfi, q)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zeros_and_what_is_not_finite(sfi, dtype):
    """A head of zeros stays zero, without eps too; an infinity is NaN after the norm, and its head's other
    elements, which it dwarfs, are 0 where its pair leaves them alone; the heads beside keep their bits."""
    q = normal((4, 6, 64), dtype, 3)
    for eps in (0.0, 1e-40, 1e-6):
        good = call(sfi, q, eps=eps, rot=32)
        x = q.clone()
        x[0, 1] = 0
        x[1, 2, 5], x[2, 0, 60], x[3, 3, 33] = float("inf"), float("nan"), float("-inf")
        x[3, 5] *= 1e30
        x[0, 4] *= 1e-30
        out = call(sfi, x, eps=eps, rot=32)
        rest = torch.ones(4, 6, dtype=torch.bool, device="cuda")
        for at in ((0, 1), (1, 2), (2, 0), (3, 3), (3, 5), (0, 4)):
            rest[at] = False
        assert torch.equal(out[rest], good[rest])
        assert (out[0, 1] == 0).all() and out[2, 0].isnan().all()
        for at, bad in (((1, 2), [5, 21]), ((3, 3), [33])):
            assert out[at].isnan().nonzero().flatten().tolist() == bad
            assert int((out[at] == 0).sum()) == 64 - len(bad)
        check(sfi, torch.stack([x[3, 5], x[3, 4]])[None], eps=eps, rot=32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_and_small_weights(sfi, dtype):
    """The norm comes before the weight: their product with the elements may leave fp32 where the output does
    not."""
    for scale, up in ((1e13, 1e30), (1e-13, 1e-33), (1e10, 1e36), (1e-14, 1e-32)):
        q = normal((3, 4, 128), F32, 1).clamp(-4.5, 4.5).mul(scale).to(dtype)
        w = (1 + 0.3 * normal((128,), F32, 5)).mul(up).to(dtype)
        for eps in (0.0, 1e-6) if scale > 1 else (0.0,):
            check(sfi, q, w, eps=eps)
            check(sfi, q, w, rot=64, interleaved=True, eps=eps)


@pytest.mark.parametrize("eps", [1e20, 1e30, 3e38])
def test_large_eps(sfi, eps):
    eps = float(np.float32(eps))
    for scale in (1e-3, 1.0, 1e15, 1e19, 1e30):
        check(sfi, normal((2, 3, 64), F32, 1).mul(scale), eps=eps)


@pytest.mark.parametrize("rows", [3, 5000])
def test_far_heads_beside_others(sfi, rows):
    """Rows with heads of all sizes, over warps or a warp a row: each row alone gives the same bits, and q and k
    of the same call may both hold such heads."""
    d, hq, hkv = 128, 7, 3
    q, k = normal((rows, hq, d), F32, 5), normal((rows, hkv, d), F32, 6)
    for x, s in ((q, 7), (k, 8)):
        g = torch.Generator().manual_seed(s)
        x *= torch.exp2(120 * (2 * torch.rand(x.shape[:2], generator=g) - 1)).cuda()[..., None]
    q, k = q.to(BF16), k.to(BF16)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    sfi.sfi_qk_norm_rope(sfi.RotaryLayout(hq, hkv, d, BF16, pos, eps=0.0), q, k, qo, ko)
    freq = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    for t in sorted({0, 1, rows // 2, rows - 1}):
        q1, k1 = torch.empty_like(q[:1]), torch.empty_like(k[:1])
        sfi.sfi_qk_norm_rope(sfi.RotaryLayout(hq, hkv, d, BF16, pos[t:t + 1], eps=0.0), q[t:t + 1], k[t:t + 1], q1, k1)
        assert torch.equal(q1[0], qo[t]) and torch.equal(k1[0], ko[t])
        for x, y in ((q, qo), (k, ko)):
            ref, size = H.norm_rope(f64(x[t:t + 1]), None, [t], freq, False, 0.0)
            close(f64(y[t:t + 1]), ref, tolerance(ref, size, BF16), "out")
