"""CPU checks of what the norm and rotation of heads and the 8-bit paged cache refuse, before any
GPU work, and of the restatements that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.heads_oracle as H
from tests.sfi_testlib import load_sfi
from tests.test_paged_abi import FAKE, paged, ref, store


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def rope(sfi, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, qo=FAKE, ko=FAKE, **kw):
    freq = (ctypes.c_double * 64)(*kw.pop("freq", [1.0] * 64))
    d = dict(total=3, n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=sfi.SFI_BF16, rotary_dim=64, interleaved=0, norm=1, eps=1e-6,
             pos_offset=0, q_stride=0, k_stride=0, q_out_stride=0, k_out_stride=0, pos=FAKE, inv_freq=ctypes.addressof(freq))
    d.update(kw)
    return sfi.lib.sfi_qk_norm_rope(ctypes.byref(sfi.sfi_rotary_layout(**d)), q, k, wq, wk, qo, ko, None)


def test_rope_refusals(sfi):
    bad, unsup, cap = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED, sfi.SFI_ERR_CAPACITY
    assert sfi.lib.sfi_qk_norm_rope(None, FAKE, FAKE, None, None, FAKE, FAKE, None) == bad
    for kw, code in [(dict(total=-1), bad), (dict(n_q_heads=-1), bad), (dict(n_q_heads=0, n_kv_heads=0), bad), (dict(n_q_heads=4097), cap),
                     (dict(n_kv_heads=5000), cap), (dict(head_dim=96), unsup), (dict(dtype=4), unsup), (dict(dtype=2), unsup),
                     (dict(rotary_dim=-8), bad), (dict(rotary_dim=72), bad), (dict(rotary_dim=12), bad), (dict(inv_freq=None), bad),
                     (dict(eps=-1.0), bad), (dict(eps=float("nan")), bad), (dict(eps=float("inf")), bad), (dict(norm=0), bad),
                     (dict(norm=0, wq=None), bad), (dict(freq=[float("inf")] * 64), bad), (dict(freq=[float("nan")] * 64), bad),
                     (dict(freq=[-2.0 ** 33] * 64), bad),
                     (dict(q_stride=511), bad), (dict(q_stride=516), bad), (dict(k_stride=64), bad), (dict(q_out_stride=-512), bad),
                     (dict(k_out_stride=132), bad), (dict(k_stride=1 << 40), cap), (dict(pos=None), bad), (dict(q=None), bad),
                     (dict(k=None), bad), (dict(qo=None), bad), (dict(ko=None), bad), (dict(q=FAKE + 8), bad), (dict(ko=FAKE + 4), bad),
                     (dict(wq=FAKE + 2), bad), (dict(q_stride=1024), bad)]:  # (q is q_out here)
        assert rope(sfi, **kw) == code, kw
    assert rope(sfi, total=0, q=None, k=None, qo=None, ko=None, pos=None) == sfi.SFI_OK


def attn8(sfi, L, q=FAKE, k=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40, dtype=1):
    return sfi.lib.sfi_paged_attn_q8(ref(L), dtype, q, k, FAKE, out, None, ws, ws_bytes, None)


def append8(sfi, L, total=4, new=FAKE, ks=0, vs=0, cu=None, k=FAKE, ws=FAKE, ws_bytes=1 << 40, dtype=1):
    return sfi.lib.sfi_paged_append_q8(ref(L), dtype, total, new, FAKE, ks, vs, cu, k, FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("dtype", [4, 5])
def test_q8_layout_refusals(sfi, dtype):
    bad, unsup, cap = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED, sfi.SFI_ERR_CAPACITY
    page = 2 * 16 * (64 + 4)
    for kw, code in [(dict(batch=0), bad), (dict(n_q_heads=9), bad), (dict(n_q_heads=34), unsup), (dict(head_dim=80), unsup),
                     (dict(page_size=0), bad), (dict(page_size=1025), cap), (dict(page_stride=page - 16), bad),
                     (dict(page_stride=page + 8), bad), (dict(page_stride=1 << 39), cap), (dict(n_pages=1 << 24, page_stride=1 << 18), cap),
                     (dict(page_table=None), bad), (dict(len=None), bad)]:
        L = paged(sfi, **{**kw, "dtype": dtype})
        assert sfi.lib.sfi_paged_workspace_size(ref(L)) == 0, kw
        assert attn8(sfi, L) == code and append8(sfi, L) == code, kw
        assert sfi.lib.sfi_pages_extend(ref(L), ref(store(sfi)), None, FAKE, 1 << 40, None) == code, kw
    assert attn8(sfi, None) == bad and append8(sfi, None) == bad
    L, plain = paged(sfi, dtype=dtype), paged(sfi)
    need = sfi.lib.sfi_paged_workspace_size(ref(L))
    assert need > 0
    # each kind of pool has its own calls
    assert attn8(sfi, plain) == unsup and append8(sfi, plain) == unsup
    assert sfi.lib.sfi_paged_attn(ref(L), FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 40, None) == unsup
    assert sfi.lib.sfi_paged_append(ref(L), 4, FAKE, FAKE, 0, 0, None, FAKE, FAKE, FAKE, 1 << 40, None) == unsup
    for t in (2, 4, 5, 9):
        assert attn8(sfi, L, dtype=t) == unsup and append8(sfi, L, dtype=t) == unsup
    for kw in (dict(q=None), dict(k=None), dict(out=None), dict(q=FAKE + 4), dict(k=FAKE + 8)):
        assert attn8(sfi, L, **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=need - 1)):
        assert attn8(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE and append8(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE, kw
    for kw in (dict(total=-1), dict(total=3), dict(new=None), dict(new=FAKE + 8), dict(k=None), dict(k=FAKE + 4), dict(ks=127),
               dict(ks=132), dict(vs=64), dict(vs=-128)):
        assert append8(sfi, L, **kw) == bad, kw
    assert append8(sfi, L, ks=132, dtype=0, total=0, cu=FAKE) == sfi.SFI_OK  # (fp32 rows: 528 bytes)
    # the bookkeeping's layers lie a multiple of 16 bytes apart
    S = store(sfi, layer_stride=1000 * 16 + 8)
    assert sfi.lib.sfi_pages_compact(ref(L), ref(S), None, FAKE, 1 << 40, None) == bad


def test_quantise_restatement_by_hand():
    c, s = H.quantise(np.array([[127.0, 63.5, -63.5, 0.5, 1.5, -127.0]]), "i8")
    assert s[0] == 1 and c[0].tolist() == [127, 64, -64, 0, 2, -127]
    c, s = H.quantise(np.array([[448.0, 1.0, 17.0, 19.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]]), "e4m3")
    assert s[0] == 1 and c[0].tolist() == [448, 1, 16, 20, 2.0 ** -9, 0, 2.0 ** -8]
    c, s = H.quantise(np.array([[448.5, 0.0]]), "e4m3")
    assert s[0] == 2 and c[0, 0] == 224
    c, s = H.quantise(np.array([[0.0, 0.0], [np.inf, 1.0]]), "i8")
    assert s[0] == 0 and np.isnan(s[1]) and (c == 0).all()


@pytest.mark.parametrize("x", [0.3, 5.0, 100.0, 400.0, 2.0 ** -8])
def test_quantise_restatement_against_the_type(x):
    """e4m3 codes are the type's own numbers, rounded as a conversion rounds them."""
    row = np.float32([448.0, x, -x, x * 1.0625, x * 1.03125])
    c, s = H.quantise(row[None], "e4m3")
    t = torch.from_numpy(row).to(torch.float8_e4m3fn).double().numpy()
    assert s[0] == 1 and np.array_equal(c[0], t)


def test_rotation_restatement_by_hand():
    x = np.zeros((2, 1, 64))
    x[:, 0, 1], x[:, 0, 4] = 3.0, 5.0
    freq = [np.pi / 2] + [0.0] * 3
    y, _ = H.norm_rope(x, None, [1, 2], freq, False, None)  # pairs (0, 4), (1, 5) ..
    assert np.allclose(y[:, 0, 4], [0, -5], atol=1e-12) and np.allclose(y[:, 0, 0], [-5, 0], atol=1e-12) and (y[:, 0, 1] == 3).all()
    y, _ = H.norm_rope(x, None, [1, 2], freq, True, None)   # pairs (0, 1), (2, 3) ..
    assert np.allclose(y[:, 0, 0], [-3, 0], atol=1e-12) and np.allclose(y[:, 0, 1], [0, -3], atol=1e-12)
    y, _ = H.norm_rope(np.full((1, 1, 64), 2.0), np.full(64, 0.5), [0], [], False, 0.0)
    assert np.allclose(y, 0.5)


def shared(sfi, L, n=1, cu=FAKE, pages=FAKE, q=FAKE, k=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return sfi.lib.sfi_paged_attn_shared(ref(L), n, cu, pages, q, k, FAKE, out, None, ws, ws_bytes, None)


def test_shared_refusals(sfi):
    bad, unsup, cap = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED, sfi.SFI_ERR_CAPACITY
    for kw, code in [(dict(batch=0), bad), (dict(head_dim=80), unsup), (dict(n_q_heads=34), unsup), (dict(dtype=0), unsup),
                     (dict(dtype=4), unsup), (dict(dtype=5), unsup), (dict(dtype=2), unsup), (dict(page_size=0), bad), (dict(len=None), bad)]:
        L = paged(sfi, **kw)
        assert shared(sfi, L) == code, kw
        assert sfi.lib.sfi_paged_shared_workspace_size(ref(L), 1) == 0, kw
    L = paged(sfi)
    size = sfi.lib.sfi_paged_shared_workspace_size
    assert shared(sfi, None) == bad and shared(sfi, L, n=-1) == bad and shared(sfi, L, n=1025) == cap
    assert size(ref(L), -1) == 0 and size(ref(L), 1025) == 0
    for kw in (dict(cu=None), dict(pages=None), dict(q=None), dict(k=None), dict(out=None), dict(q=FAKE + 8), dict(k=FAKE + 2), dict(out=FAKE + 4)):
        assert shared(sfi, L, **kw) == bad, kw
    need = size(ref(L), 1)
    assert need > size(ref(L), 0) >= sfi.lib.sfi_paged_workspace_size(ref(L)) > 0
    assert size(ref(L), 1024) >= size(ref(L), 2) >= need
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=need - 1)):
        assert shared(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE, kw
