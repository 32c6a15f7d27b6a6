"""CPU checks of the prompt attention's and the paged cache's host-side refusals: bad arguments
are named before any GPU work."""
import ctypes

import pytest
import torch

from tests.sfi_testlib import load_sfi

FAKE = 0x10000  # never dereferenced: every call below fails host validation first


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def packed(sfi, **kw):
    d = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=sfi.SFI_BF16, total_q=100, total_k=100,
             q_stride=0, k_stride=0, v_stride=0, out_stride=0, cu_q=FAKE, cu_k=FAKE)
    d.update(kw)
    return sfi.sfi_packed_layout(**d)


def prefill(sfi, L, q=FAKE, k=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 20):
    return sfi.lib.sfi_prefill_attn(ctypes.byref(L) if L is not None else None, q, k, FAKE, out, None, ws, ws_bytes, None)


def test_prefill_refusals(sfi):
    bad, unsup = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED
    assert prefill(sfi, None) == bad
    for kw, code in [(dict(batch=0), bad), (dict(batch=1025), sfi.SFI_ERR_CAPACITY), (dict(n_q_heads=7), bad),
                     (dict(n_kv_heads=0), bad), (dict(n_q_heads=34), unsup), (dict(head_dim=96), unsup),
                     (dict(dtype=sfi.SFI_F32), unsup), (dict(dtype=9), unsup), (dict(total_q=-1), bad),
                     (dict(total_k=-1), bad), (dict(cu_q=None), bad), (dict(cu_k=None), bad),
                     (dict(q_stride=511), bad), (dict(q_stride=516), bad), (dict(k_stride=64), bad),
                     (dict(v_stride=-128), bad), (dict(out_stride=500), bad),
                     (dict(k_stride=1 << 40), sfi.SFI_ERR_CAPACITY),
                     (dict(total_q=2**31 - 1, n_q_heads=1600, n_kv_heads=100), sfi.SFI_ERR_CAPACITY)]:
        assert prefill(sfi, packed(sfi, **kw)) == code, kw
    L = packed(sfi)
    assert prefill(sfi, L, q=None) == bad and prefill(sfi, L, k=None) == bad and prefill(sfi, L, out=None) == bad
    assert prefill(sfi, L, q=FAKE + 8) == bad and prefill(sfi, L, out=FAKE + 2) == bad
    for kw in (dict(ws=None), dict(ws_bytes=255), dict(ws=FAKE + 16)):
        assert prefill(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE
    assert sfi.lib.sfi_prefill_attn_workspace_size(ctypes.byref(L)) > 0
    assert sfi.lib.sfi_prefill_attn_workspace_size(ctypes.byref(packed(sfi, head_dim=32))) == 0
    # nothing to compute: no pointer is needed
    assert prefill(sfi, packed(sfi, total_q=0), q=None, k=None, out=None) == sfi.SFI_OK


def test_binding_refuses_host_tensors(sfi):
    cu = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        sfi.PackedLayout(8, 2, 64, torch.bfloat16, cu, cu, 10, 10)
