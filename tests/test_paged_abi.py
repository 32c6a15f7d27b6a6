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


def paged(sfi, **kw):
    d = dict(batch=4, n_q_heads=8, n_kv_heads=2, head_dim=64, dtype=sfi.SFI_BF16, page_size=16, n_pages=100,
             max_pages=20, page_stride=0, page_table=FAKE, len=FAKE)
    d.update(kw)
    return sfi.sfi_paged_layout(**d)


def store(sfi, **kw):
    d = dict(ref=FAKE, k=FAKE, v=FAKE, n_layers=2, layer_stride=1 << 20)
    d.update(kw)
    return sfi.sfi_page_store(**d)


def ref(x):
    return ctypes.byref(x) if x is not None else None


def attn(sfi, L, q=FAKE, k=FAKE, out=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return sfi.lib.sfi_paged_attn(ref(L), q, k, FAKE, out, None, ws, ws_bytes, None)


def append(sfi, L, total=4, new=FAKE, ks=0, vs=0, cu=None, k=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return sfi.lib.sfi_paged_append(ref(L), total, new, FAKE, ks, vs, cu, k, FAKE, ws, ws_bytes, None)


def arr(v):
    return (ctypes.c_int32 * max(1, len(v)))(*v)


def test_paged_layout_refusals(sfi):
    bad, unsup, cap = sfi.SFI_ERR_INVALID_ARG, sfi.SFI_ERR_UNSUPPORTED, sfi.SFI_ERR_CAPACITY
    for kw, code in [(dict(batch=0), bad), (dict(batch=1025), cap), (dict(batch=1024, n_q_heads=5, n_kv_heads=5), cap),
                     (dict(n_q_heads=9), bad), (dict(n_q_heads=34), unsup), (dict(head_dim=80), unsup),
                     (dict(dtype=2), unsup), (dict(page_size=0), bad), (dict(page_size=1025), cap),
                     (dict(n_pages=0), bad), (dict(n_pages=(1 << 24) + 1), cap), (dict(max_pages=0), bad),
                     (dict(max_pages=1 << 27), cap), (dict(page_stride=2047), bad), (dict(page_stride=2080), bad),
                     (dict(page_stride=-2048), bad), (dict(page_stride=1 << 39), cap),
                     (dict(n_pages=1 << 20, page_stride=1 << 18), cap),
                     (dict(batch=1, n_q_heads=4096, n_kv_heads=4096, page_size=1024, head_dim=128), cap),
                     (dict(page_table=None), bad), (dict(len=None), bad)]:
        L = paged(sfi, **kw)
        assert sfi.lib.sfi_paged_workspace_size(ref(L)) == 0, kw
        assert attn(sfi, L) == code and append(sfi, L) == code, kw
        assert sfi.lib.sfi_pages_extend(ref(L), ref(store(sfi)), None, FAKE, 1 << 40, None) == code, kw
    assert attn(sfi, None) == bad and append(sfi, None) == bad
    need = sfi.lib.sfi_paged_workspace_size(ref(paged(sfi)))
    assert need > 0 and sfi.lib.sfi_paged_workspace_size(ref(paged(sfi, n_pages=10000))) > need


def test_paged_attn_and_append_refusals(sfi):
    bad, L = sfi.SFI_ERR_INVALID_ARG, paged(sfi)
    need = sfi.lib.sfi_paged_workspace_size(ref(L))
    for kw in (dict(q=None), dict(k=None), dict(out=None), dict(q=FAKE + 4), dict(k=FAKE + 8)):
        assert attn(sfi, L, **kw) == bad, kw
    for kw in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=need - 1)):
        assert attn(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE and append(sfi, L, **kw) == sfi.SFI_ERR_WORKSPACE, kw
    for kw in (dict(total=-1), dict(total=3), dict(new=None), dict(new=FAKE + 8), dict(k=None), dict(k=FAKE + 4),
               dict(ks=127), dict(ks=132), dict(vs=64), dict(vs=-128)):
        assert append(sfi, L, **kw) == bad, kw
    assert append(sfi, L, total=0, cu=FAKE, new=None) == sfi.SFI_OK  # nothing to store


def test_page_call_refusals(sfi):
    bad, L, S = sfi.SFI_ERR_INVALID_ARG, paged(sfi), store(sfi)

    def fork(src, dst, n=None, S=S, ws=FAKE):
        return sfi.lib.sfi_pages_fork(ref(L), ref(S), arr(src) if src is not None else None, arr(dst),
                                      len(dst) if n is None else n, ws, 1 << 40, None)

    def free(seqs, n=None, S=S, ws=FAKE):
        return sfi.lib.sfi_pages_free(ref(L), ref(S), arr(seqs) if seqs is not None else None,
                                      len(seqs) if n is None else n, ws, 1 << 40, None)

    def copy(n, src=FAKE, S=S, ws=FAKE):
        return sfi.lib.sfi_pages_copy(ref(L), ref(S), src, FAKE, n, ws, 1 << 40, None)

    def compact(S=S, ws=FAKE):
        return sfi.lib.sfi_pages_compact(ref(L), ref(S), None, ws, 1 << 40, None)

    def extend(S=S, ws=FAKE):
        return sfi.lib.sfi_pages_extend(ref(L), ref(S), None, ws, 1 << 40, None)

    for src, dst in (([0], [4]), ([-1], [1]), ([0, 0], [1, 1]), ([0, 1], [1, 2]), ([2], [2])):
        assert fork(src, dst) == bad, (src, dst)
    assert fork(None, [1], n=1) == bad and fork([0], [1], n=-1) == bad and fork([0] * 5, [1, 2, 3, 0, 1], n=5) == bad
    assert free([0, 0]) == bad and free([4]) == bad and free([-1]) == bad and free(None, n=1) == bad
    assert copy(-1) == bad and copy(101) == bad and copy(1, src=None) == bad
    for S2 in (None, store(sfi, ref=None)):
        assert bad == fork([0], [1], S=S2) == free([0], S=S2) == copy(1, S=S2) == compact(S=S2) == extend(S=S2)
    for kw, code in [(dict(k=None), bad), (dict(v=FAKE + 8), bad), (dict(n_layers=0), bad), (dict(layer_stride=0), bad),
                     (dict(layer_stride=-64), bad), (dict(layer_stride=96), bad),
                     (dict(n_layers=5000), sfi.SFI_ERR_CAPACITY), (dict(layer_stride=1 << 42), sfi.SFI_ERR_CAPACITY)]:
        S2 = store(sfi, **kw)
        assert code == fork([0], [1], S=S2) == copy(1, S=S2) == compact(S=S2), kw
    w = sfi.SFI_ERR_WORKSPACE
    assert w == fork([0], [1], ws=None) == free([0], ws=None) == copy(1, ws=None) == compact(ws=None) == extend(ws=None)
    assert fork([], []) == free([]) == copy(0) == sfi.SFI_OK  # nothing to do


def test_binding_refuses_mismatched_pools(sfi):
    with pytest.raises(ValueError):
        sfi.PagedLayout(8, 2, 64, torch.bfloat16, 16, 10, torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    k = torch.zeros(3, 2, 16, 64)
    with pytest.raises(ValueError):
        sfi.PageStore(torch.zeros(3, dtype=torch.int32), k, k[:2])


def test_binding_refuses_rows_that_overlap(sfi):
    """A stride of 0 means rows without gaps to the C calls: an expanded row is none of that."""
    row, shape = torch.zeros(1, 2, 64), (3, 2, 64)
    flat = torch.zeros(1000)
    for t in (row.expand(shape), flat.as_strided(shape, (64, 64, 1)), flat.as_strided(shape, (127, 64, 1))):
        with pytest.raises(ValueError):
            sfi._want("q", t, shape, torch.float32, t.device, True)
    for t, n in ((row.expand(1, 2, 64), 1), (flat.as_strided(shape, (192, 64, 1)), 3), (torch.zeros(0, 2, 64), 0)):
        sfi._want("q", t, (n, 2, 64), torch.float32, t.device, True)
