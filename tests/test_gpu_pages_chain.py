"""Extending sequences and storing their rows in a row, without a look at the status between, as a
decode step does it: where pages run out, the rows of a refused sequence go nowhere."""
import numpy as np
import pytest
import torch

from tests.paged_testlib import f64, ints, normal, offsets
from tests.sfi_testlib import load_sfi
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


class Chain(Pool):
    """The restatement stores the rows of the sequences that the last extension did not refuse."""

    def model_step(self, n, kn, vn, layer):
        """Extend by n, then n rows a sequence; returns the flags of the two calls."""
        m = self.model
        old, cu = m.len.copy(), offsets(n)
        flags = set(m.extend(n))
        own, rows = [0], []
        for b, x in enumerate(n):
            if x > 0 and m.len[b] == old[b] + x:
                rows += range(cu[b], cu[b + 1])
            own.append(len(rows))
        m.append(layer, kn[rows], vn[rows], own)
        return flags

    def rows(self, n, seed):
        shape = (n,) + tuple(self.k.shape[i] for i in (2, 4))
        return normal(shape, self.k.dtype, seed), normal(shape, self.k.dtype, seed + 1)

    def step(self, n, seed, layer=0, between=None):
        cu = offsets(n)
        kn, vn = self.rows(cu[-1], seed)
        self.sfi.sfi_pages_extend(self.lay, self.store, ints(n), self.ws)
        if between:
            between()
        self.sfi.sfi_paged_append(self.lay, kn, vn, self.k[layer], self.v[layer], ints(cu), self.ws)
        self.same(self.model_step(n, f64(kn), f64(vn), layer))

    def token(self, seed, flags):
        """The decode step's form: a row for each sequence, idle slots among them."""
        B = len(self.model.len)
        kn, vn = self.rows(B, seed)
        self.sfi.sfi_pages_extend(self.lay, self.store, None, self.ws)
        self.sfi.sfi_paged_append(self.lay, kn, vn, self.k[0], self.v[0], None, self.ws)
        n = [int(x > 0) for x in self.model.len]
        live = [b for b in range(B) if n[b]]
        assert self.model_step(n, f64(kn)[live], f64(vn)[live], 0) == set(flags)
        self.same(flags)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_refused_fork_keeps_the_shared_page(sfi, dtype):
    """Two forks share two full pages of 4 and no page is free: each needs one for its token."""
    p = Chain(sfi, 2, 64, dtype, 4, [8, 0], 0, width=5)
    p.fork([0], [1])
    p.token(20, ["pages"])
    p.token(22, ["pages"])
    p.step([1, 1], 24, layer=1)
    p.step([3, 2], 26)
    assert p.model.len.tolist() == [8, 8]


def test_refused_until_served(sfi):
    """Some are refused and some served in one call; a freed sequence's pages serve the refused."""
    p = Chain(sfi, 2, 64, BF16, 4, [8, 6, 3, 12, 0], 1, width=6)
    p.token(20, ["pages"])             # 0 takes the free page, 1 and 2 have room, 3 is refused
    assert p.model.len.tolist() == [9, 7, 4, 12, 0]
    p.step([1, 0, 2, 0, 3], 22)        # 2 and 4 find none
    assert p.model.len.tolist() == [10, 7, 4, 12, 0]
    p.free([1])
    p.step([0, 0, 2, 0, 3], 24)
    assert p.model.len.tolist() == [10, 0, 6, 12, 3]
    p.step([2, 0, 2, 0, 1], 26)
    p.free([3])
    p.step([1, 1, 0, 2, 0], 28)
    p.token(30, ["pages"])            # no page is left again: 2 and 4 are refused
    p.held_counts_match()


def test_refused_chunk(sfi):
    """A chunk of a long prompt that finds too few pages does not go over the last chunk."""
    p = Chain(sfi, 2, 128, BF16, 16, [700, 40], 40, width=80)
    p.step([500, 500], 20)             # the second finds too few
    assert p.model.len.tolist() == [1200, 40]
    p.step([600, 900], 22)
    p.step([1, 1], 24)


def test_refused_for_other_reasons(sfi):
    """A full row of the table, negative growth: left out of the append as well."""
    p = Chain(sfi, 1, 64, BF16, 4, [12, 5, 11], 9, width=3)
    p.step([1, 2, 1], 20)              # the first one's row holds 3 pages
    p.step([4, 0, 1], 22)
    kn, vn = p.rows(3, 24)
    sfi.sfi_pages_extend(p.lay, p.store, ints([0, -1, 0]), p.ws)
    sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], ints([0, 0, 2, 2]), p.ws)
    p.same(["len", "pages"])
    p.free([0, 1])
    p.step([3, 12, 0], 26)
    p.held_counts_match()


def test_fork_into_a_refused_slot(sfi):
    """A slot whose prompt was refused takes a fork; rows may then be stored there again."""
    p = Chain(sfi, 1, 64, BF16, 4, [6, 0], 1, width=4)
    p.step([0, 9], 20)
    p.fork([0], [1])
    kn, vn = p.rows(2, 22)             # over its own last rows: no extension between
    sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], ints([0, 0, 2]), p.ws)
    p.model.append(0, f64(kn), f64(vn), [0, 0, 2])
    p.same()


def test_appends_without_an_extension(sfi):
    """Lengths set by the caller and a workspace that saw no refusal: everything is stored; so it
    is again after the workspace was zero-filled."""
    p = Chain(sfi, 1, 64, BF16, 4, [8, 3], 0)
    p.append(0, [5, 2])
    p.step([1, 1], 20)
    p.ws.zero_()
    p.append(1, [1, 1])


def test_largest_batch(sfi):
    """Every bit of the refused: 1024 sequences, of which every third needs a page and few get one."""
    lens = [4 if b % 3 == 0 else 3 for b in range(1024)]
    p = Chain(sfi, 1, 64, BF16, 4, lens, 100, layers=1, width=3)
    p.step([1] * 1024, 20)
    assert int((p.model.len == 5).sum()) == 100
    gone = [b for b in range(1024) if b % 3 == 1]
    p.free(gone)
    p.step([int(b % 3 != 1) for b in range(1024)], 22)


def test_prompt_attention_between(sfi):
    """The prompt attention on the same workspace, between the two calls, leaves the refusals alone."""
    hq, hkv, d, lens = 8, 2, 64, [1500, 300, 77]
    cu = offsets(lens)
    q, k = normal((cu[-1], hq, d), BF16, 1), normal((cu[-1], hkv, d), BF16, 2)
    prompts = sfi.PackedLayout(hq, hkv, d, BF16, ints(cu), ints(cu), cu[-1], cu[-1])
    out = torch.empty_like(q)
    p = Chain(sfi, 2, 64, BF16, 4, [8, 4], 0, width=5)
    n = max(p.ws.numel(), sfi.prefill_workspace(prompts).numel())
    p.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    p.step([1, 1], 20, between=lambda: sfi.sfi_prefill_attn(prompts, q, k, k, out, None, p.ws))


def test_captured_until_the_pages_run_out(sfi):
    """A captured step replayed past the last free page: nothing can look at the status between."""
    p = Chain(sfi, 2, 64, BF16, 4, [6, 3, 0, 8], 3, width=9)
    p.fork([3], [2])
    kn, vn = p.rows(4, 20)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            sfi.sfi_pages_extend(p.lay, p.store, None, p.ws)
            sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], None, p.ws)
        for _ in range(9):
            g.replay()
        st.synchronize()
    flags = set()
    for _ in range(9):
        flags |= p.model_step([1] * 4, f64(kn), f64(vn), 0)
    assert flags == {"pages"} and p.model.len.max() < 15
    p.same(flags)
    p.held_counts_match()
