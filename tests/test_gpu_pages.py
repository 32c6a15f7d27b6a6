"""Storing rows in pages and the page bookkeeping against the restatement that moves one page at
a time: results are integers and moved values, so everything is compared exactly."""
import random

import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import bf16_tolerance, close, f32_tolerance, f64, ints, normal, offsets, pool_of
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


class Pool:
    """A cache on the device and the same one in the restatement."""

    def __init__(self, sfi, hkv, d, dtype, page, lens, extra, layers=2, seed=1, width=0):
        self.sfi = sfi
        n_pages, rows = pool_of(lens, page, extra, seed)
        if width > rows.shape[1]:
            rows = np.pad(rows, ((0, 0), (0, width - rows.shape[1])), constant_values=-1)
        ref = np.zeros(n_pages, np.int32)
        ref[rows[rows >= 0]] = 1
        shape = (layers, n_pages, hkv, page, d)
        self.k, self.v = normal(shape, dtype, seed + 1), normal(shape, dtype, seed + 2)
        self.table, self.len, self.ref = ints(rows.tolist()), ints(list(lens)), ints(ref.tolist())
        self.model = P.Pages(rows, lens, ref, f64(self.k), f64(self.v))
        self.lay = sfi.PagedLayout(hkv, hkv, d, dtype, page, n_pages, self.table, self.len)
        self.store = sfi.PageStore(self.ref, self.k, self.v)
        self.ws = sfi.paged_workspace(self.lay)

    def same(self, flags=()):
        names = {"pages": self.sfi.SFI_DEV_NO_PAGES, "index": self.sfi.SFI_DEV_BAD_INDEX, "len": self.sfi.SFI_DEV_LEN_OVER_CAP}
        assert self.sfi.sfi_read_status(self.ws) == sum(names[x] for x in flags)
        m = self.model
        assert np.array_equal(f64(self.len), m.len) and np.array_equal(f64(self.ref), m.ref)
        assert np.array_equal(f64(self.table), m.table)
        assert np.array_equal(f64(self.k), m.k, equal_nan=True) and np.array_equal(f64(self.v), m.v, equal_nan=True)

    def held_counts_match(self):
        ref = np.zeros(len(self.model.ref), int)
        for b in range(len(self.model.len)):
            for i in range(self.model.held(b)):
                ref[self.model.table[b, i]] += 1
        assert np.array_equal(ref, self.model.ref)

    def extend(self, n):
        self.sfi.sfi_pages_extend(self.lay, self.store, ints(n), self.ws)
        self.same(self.model.extend(n))

    def fork(self, src, dst):
        self.sfi.sfi_pages_fork(self.lay, self.store, src, dst, self.ws)
        self.same(self.model.fork(src, dst))

    def free(self, seqs):
        self.sfi.sfi_pages_free(self.lay, self.store, seqs, self.ws)
        self.same(self.model.free(seqs))

    def compact(self):
        ids = torch.full((len(self.model.ref),), 77, dtype=torch.int32, device="cuda")
        self.sfi.sfi_pages_compact(self.lay, self.store, ids, self.ws)
        assert np.array_equal(f64(ids), self.model.compact())
        self.same()

    def append(self, layer, m, seed=9):
        cu = offsets(m)
        shape = (cu[-1],) + tuple(self.k.shape[i] for i in (2, 4))
        kn, vn = normal(shape, self.k.dtype, seed), normal(shape, self.k.dtype, seed + 1)
        self.sfi.sfi_paged_append(self.lay, kn, vn, self.k[layer], self.v[layer], ints(cu), self.ws)
        self.model.append(layer, f64(kn), f64(vn), cu)
        self.same()


@pytest.mark.parametrize("hkv,d,dtype,page", [(2, 128, BF16, 16), (3, 64, BF16, 5), (1, 64, F32, 1), (8, 128, F32, 20)])
def test_append(sfi, hkv, d, dtype, page):
    p = Pool(sfi, hkv, d, dtype, page, [1, 40, 0, 17, page, 3], 2)
    p.append(1, [1, 33, 0, 17, 1, 2])
    p.append(0, [0, 0, 0, 0, 0, 1])
    p.append(0, [0] * 6)
    # one row per sequence; the idle slot's row goes nowhere
    kn, vn = normal((6, hkv, d), dtype, 5), normal((6, hkv, d), dtype, 6)
    p.sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], None, p.ws)
    keep = [0, 1, 3, 4, 5]
    p.model.append(0, f64(kn)[keep], f64(vn)[keep], [0, 1, 2, 2, 3, 4, 5])
    p.same()


def test_append_strided_and_longest(sfi):
    """Rows as slices of one projection; a prompt of many tokens; rows behind the last sequence."""
    hkv, d = 2, 64
    p = Pool(sfi, hkv, d, BF16, 16, [5000, 30], 2, layers=1)
    both = normal((5040, 2 * hkv * d + 24), BF16, 3)
    kn, vn = (both[:, 8 + i * hkv * d:8 + (i + 1) * hkv * d].view(-1, hkv, d) for i in (0, 1))
    cu = [3, 5003, 5030]
    sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], ints(cu), p.ws)
    p.model.append(0, f64(kn), f64(vn), cu)
    p.same()


def test_append_flags(sfi):
    """More rows than positions, descending or overlong offsets, a page outside the pool: flagged
    and left out, the other sequences are stored."""
    for cu, lens, flag, stored in (([0, 3, 9], [2, 6], "len", [1]), ([0, 5, 4], [8, 8], "len", [0]),
                                   ([0, 4, 11], [8, 8], "len", [0]), ([-1, 4, 9], [8, 8], "len", [1])):
        p = Pool(sfi, 2, 64, BF16, 4, lens, 1)
        kn, vn = normal((10, 2, 64), BF16, 5), normal((10, 2, 64), BF16, 6)
        sfi.sfi_paged_append(p.lay, kn, vn, p.k[0], p.v[0], ints(cu), p.ws)
        for b in stored:
            own = [0, 0, 0]
            own[b + 1:] = [cu[b + 1] - cu[b]] * (2 - b)
            p.model.append(0, f64(kn)[cu[b]:], f64(vn)[cu[b]:], own)
        p.same([flag])
    p = Pool(sfi, 2, 64, BF16, 4, [8, 8], 1)
    for bad in (p.lay.n_pages, -1):
        p.table[0, 1] = p.model.table[0, 1] = bad
        kn = normal((2, 2, 64), BF16, 5)
        sfi.sfi_paged_append(p.lay, kn, kn, p.k[0], p.v[0], None, p.ws)
        p.model.append(0, f64(kn)[1:], f64(kn)[1:], [0, 0, 1])
        p.same(["index"])


def test_extend(sfi):
    p = Pool(sfi, 1, 64, BF16, 8, [0, 7, 8, 9, 30], 20, width=12)
    p.extend([1, 1, 1, 1, 1])
    p.extend([0, 20, 0, 40, 3])
    p.extend([0, 0, 0, 0, 0])
    sfi.sfi_pages_extend(p.lay, p.store, None, p.ws)
    p.same(p.model.extend([1] * 5))
    p.free([0])
    sfi.sfi_pages_extend(p.lay, p.store, None, p.ws)  # the empty slot stays empty
    p.same(p.model.extend([0, 1, 1, 1, 1]))
    p.held_counts_match()


def test_extend_shortage(sfi):
    """Too few pages: in order, whoever fits; a row that is full; negative growth."""
    p = Pool(sfi, 1, 64, BF16, 4, [4, 4, 4, 4, 3, 4], 3, width=6)
    p.extend([4, 12, 8, 1, 1, 0])      # 1, 3 (too many), 2, 1 (none left), 0, 0
    p.extend([0, 1, 0, 0, 0, 0])       # nothing left
    p = Pool(sfi, 1, 64, BF16, 4, [4, 4, 4], 9, width=3)
    p.extend([9, 8, -1])               # past the row's 3 entries; exactly full; negative
    p.extend([1 << 30, 0, 2])
    p.held_counts_match()


def test_large_pool_and_row(sfi):
    """Pages to be found far behind the first few thousand, and one sequence taking most of them."""
    p = Pool(sfi, 1, 64, BF16, 1, [9000, 0, 2], 5000, layers=1, width=14000)
    p.extend([0, 4990, 5])
    p.free([0])
    p.extend([0, 8000, 1000])
    p.compact()
    p.held_counts_match()


@pytest.mark.parametrize("hkv,d,dtype,page,layers", [(2, 128, BF16, 16, 3), (1, 64, F32, 5, 1), (3, 128, F32, 64, 2), (2, 64, BF16, 1, 2)])
def test_fork(sfi, hkv, d, dtype, page, layers):
    p = Pool(sfi, hkv, d, dtype, page, [page * 3 + 2, 0, 0, page, 1, 0, 0], 6, layers)
    p.fork([0, 0, 3, 4], [2, 1, 5, 6])
    p.held_counts_match()
    p.free([0, 3])
    p.fork([2], [0])
    p.fork([], [])
    p.held_counts_match()


def test_fork_refusals_on_the_device(sfi):
    """No page left for a copy, a destination that holds something, an empty source."""
    p = Pool(sfi, 1, 64, BF16, 4, [5, 0, 0, 0, 8, 0, 0], 2)
    p.fork([0, 0, 0, 4], [1, 2, 3, 6])  # the third copy finds no page; full pages need none
    p.held_counts_match()
    p.fork([0, 5], [4, 3])              # 4 is not empty; nothing of nothing
    p.len[0] = p.model.len[0] = -3
    sfi.sfi_pages_fork(p.lay, p.store, [0], [3], p.ws)
    p.same(["len"])


def test_free(sfi):
    p = Pool(sfi, 1, 64, BF16, 4, [5, 9, 0, 16], 1)
    p.free([3, 2, 0])
    p.free([0])                # empty already
    p.ref[int(p.model.table[1, 1])] = 0
    p.model.ref[p.model.table[1, 1]] = 0
    p.free([1])                # one of its pages was counted free: flagged, stays 0
    p = Pool(sfi, 1, 64, BF16, 4, [5, 9], 1)
    p.table[0, 1] = 1 << 24
    sfi.sfi_pages_free(p.lay, p.store, [0], p.ws)
    p.model.ref[p.model.table[0, 0]] -= 1
    p.model.table[0, :2] = -1
    p.model.len[0] = 0
    p.same(["index"])
    p.len[1] = p.model.len[1] = 1 << 30
    sfi.sfi_pages_free(p.lay, p.store, [1], p.ws)
    p.same(["len"])


@pytest.mark.parametrize("hkv,d,dtype,page,layers", [(2, 128, BF16, 16, 3), (1, 64, F32, 5, 1), (8, 128, F32, 64, 1), (1, 64, BF16, 1, 2)])
def test_compact(sfi, hkv, d, dtype, page, layers):
    p = Pool(sfi, hkv, d, dtype, page, [page * 3 + 2, 0, 7 * page, page, 1], 9, layers)
    p.free([0])
    p.fork([2], [0])
    p.compact()
    p.held_counts_match()
    p.compact()  # nothing to move
    p.free([0, 1, 2, 3, 4])
    p.compact()  # nothing in use


def test_compact_keeps_other_holders(sfi):
    """A page held outside the table moves too, and new_id says where it went."""
    p = Pool(sfi, 1, 64, BF16, 4, [9, 4], 5)
    x = int(np.nonzero(p.model.ref == 0)[0][-1])
    p.ref[x] = p.model.ref[x] = 3
    p.compact()


def test_compact_flags_bad_entries(sfi):
    p = Pool(sfi, 1, 64, BF16, 4, [9, 4], 5)
    p.table[0, 1] = -2
    sfi.sfi_pages_compact(p.lay, p.store, None, p.ws)
    kept = p.model.table[0, 1]
    p.model.compact()
    p.model.table[0, 1] = -2
    p.same(["index"])
    assert kept >= 0


def test_copy(sfi):
    p = Pool(sfi, 3, 64, F32, 20, [200], 30)
    src, dst = [0, 5, 5, 9, 20], [30, 31, 32, 9, 33]
    sfi.sfi_pages_copy(p.lay, p.store, ints(src), ints(dst), p.ws)
    for pool in (p.model.k, p.model.v):
        pool[:, dst] = pool[:, src]
    p.same()
    sfi.sfi_pages_copy(p.lay, p.store, ints([1, 1, -1]), ints([34, 40, 2]), p.ws)
    for pool in (p.model.k, p.model.v):
        pool[:, 34] = pool[:, 1]
    p.same(["index"])
    sfi.sfi_pages_copy(p.lay, p.store, ints([]), ints([]), p.ws)
    p.same()


def test_random_runs(sfi):
    """Long random runs of every call, compared after each."""
    r = random.Random(4)
    for page, dtype in ((4, BF16), (7, F32)):
        p = Pool(sfi, 2, 64, dtype, page, [r.randrange(40) for _ in range(9)], 25, 2, width=16)
        for step in range(40):
            what = r.choice(["extend", "extend", "fork", "free", "compact", "append"])
            empty = [b for b in range(9) if p.model.len[b] == 0]
            full = [b for b in range(9) if p.model.len[b] > 0]
            if what == "extend":
                p.extend([r.choice([0, 1, 1, 5]) for _ in range(9)])
            elif what == "fork" and empty and full:
                p.fork([r.choice(full) for _ in empty], empty)
            elif what == "free" and full:
                p.free(r.sample(full, r.randint(1, min(3, len(full)))))
            elif what == "compact":
                p.compact()
            elif what == "append":
                # (only rows of the last, unshared page)
                m = [min(int(n % page), r.randrange(4)) for n in p.model.len]
                if sum(m):
                    p.append(r.randrange(2), m, seed=step)
        p.held_counts_match()


def test_captured(sfi):
    """A decode step's bookkeeping as a graph: extend, store, free and fork, replayed."""
    p = Pool(sfi, 2, 64, BF16, 4, [6, 3, 0], 20, width=9)
    kn, vn = normal((3, 2, 64), BF16, 5), normal((3, 2, 64), BF16, 6)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            sfi.sfi_pages_extend(p.lay, p.store, None, p.ws)
            sfi.sfi_paged_append(p.lay, kn, vn, p.k[1], p.v[1], None, p.ws)
            sfi.sfi_pages_free(p.lay, p.store, [2], p.ws)
            sfi.sfi_pages_fork(p.lay, p.store, [0], [2], p.ws)
            sfi.sfi_pages_compact(p.lay, p.store, None, p.ws)
        for _ in range(5):
            g.replay()
        st.synchronize()
    for _ in range(5):
        more = [int(n > 0) for n in p.model.len]
        p.model.extend(more)
        p.model.append(1, f64(kn)[np.array(more) > 0], f64(vn)[np.array(more) > 0], offsets(more))
        p.model.free([2])
        p.model.fork([0], [2])
        p.model.compact()
    p.same()
    p.held_counts_match()


@pytest.mark.parametrize("page", [16, 20])
def test_prompt_to_tokens(sfi, page):
    """What a server does: prompts through the prompt attention, their rows into pages, tokens
    decoded, a sequence forked and another finished, the pool compacted, and on."""
    hq, hkv, d, lens, M = 8, 2, 128, [37, 64, 5, 0], 16
    n_pages = 40
    table, length = torch.full((4, M), -1, dtype=torch.int32, device="cuda"), ints([0] * 4)
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    k, v = (torch.full((n_pages, hkv, page, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    lay = sfi.PagedLayout(hq, hkv, d, BF16, page, n_pages, table, length)
    store, ws = sfi.PageStore(ref, k, v), sfi.paged_workspace(lay)
    cu = offsets(lens)
    q, kn, vn = normal((cu[-1], hq, d), BF16, 1), normal((cu[-1], hkv, d), BF16, 2), normal((cu[-1], hkv, d), BF16, 3)
    prompts = sfi.PackedLayout(hq, hkv, d, BF16, ints(cu), ints(cu), cu[-1], cu[-1])
    out = torch.empty_like(q)
    sfi.sfi_prefill_attn(prompts, q, kn, vn, out, None, ws)
    sfi.sfi_pages_extend(lay, store, ints(lens), ws)
    sfi.sfi_paged_append(lay, kn, vn, k, v, ints(cu), ws)
    r, _, scale, size = P.prefill(f64(q), f64(kn), f64(vn), cu, cu)
    close(f64(out), r, bf16_tolerance(r, scale, size, d), "prompt")
    K = [f64(kn)[cu[b]:cu[b + 1]] for b in range(4)]  # what each sequence has seen
    V = [f64(vn)[cu[b]:cu[b + 1]] for b in range(4)]
    # the prompt's last row is the first token's attention
    last = torch.stack([q[cu[b + 1] - 1] if lens[b] else q[0] for b in range(4)])
    o = torch.empty(4, hq, d, device="cuda")
    sfi.sfi_paged_attn(lay, last, k, v, o, None, ws)
    for b in range(3):
        i = cu[b + 1] - 1
        tol = bf16_tolerance(r, scale, size, d)[i] + f32_tolerance(r, scale, size, d, 64, True)[i]
        close(f64(o)[b], f64(out)[i], tol, "last row")
    for step in range(24):
        if step == 7:
            sfi.sfi_pages_fork(lay, store, [1], [3], ws)
            K[3], V[3] = K[1], V[1]
        if step == 12:
            sfi.sfi_pages_free(lay, store, [0], ws)
            K[0], V[0] = K[0][:0], V[0][:0]
        if step == 15:
            sfi.sfi_pages_compact(lay, store, None, ws)
        kt, vt, qt = normal((4, hkv, d), BF16, 50 + step), normal((4, hkv, d), BF16, 90 + step), normal((4, hq, d), BF16, step)
        sfi.sfi_pages_extend(lay, store, None, ws)
        sfi.sfi_paged_append(lay, kt, vt, k, v, None, ws)
        sfi.sfi_paged_attn(lay, qt, k, v, o, None, ws)
        for b in range(4):
            if len(K[b]):
                K[b], V[b] = np.concatenate([K[b], f64(kt)[b:b + 1]]), np.concatenate([V[b], f64(vt)[b:b + 1]])
            for h in range(hq):
                a, _, sc, sz = P.attend(f64(qt)[b, h], K[b][:, h // 4], V[b][:, h // 4], len(K[b]))
                close(f64(o)[b, h], a, f32_tolerance(a, sc, np.array(sz), d, 100, True), f"step {step}")
    assert sfi.sfi_read_status(ws) == 0


def test_one_workspace_for_prompts_and_tokens(sfi):
    """Prompt attention and paged calls in turn on one workspace: neither spoils the other's."""
    hq, hkv, d, page, lens = 8, 2, 128, 16, [3000, 700]
    cu = offsets([400, 900, 37])
    q, kn = normal((cu[-1], hq, d), BF16, 1), normal((cu[-1], hkv, d), BF16, 2)
    prompts = sfi.PackedLayout(hq, hkv, d, BF16, ints(cu), ints(cu), cu[-1], cu[-1])
    n_pages = sum(-(-n // page) for n in lens)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    rows = torch.full((2, 200), -1, dtype=torch.int32, device="cuda")
    rows[0, :188], rows[1, :44] = table[:188], table[188:]
    lay = sfi.PagedLayout(hq, hkv, d, BF16, page, n_pages, rows, ints(lens))
    k, v = normal((n_pages, hkv, page, d), BF16, 3), normal((n_pages, hkv, page, d), BF16, 4)
    own = sfi.prefill_workspace(prompts), sfi.paged_workspace(lay)
    both = torch.zeros(max(x.numel() for x in own), dtype=torch.uint8, device="cuda")
    outs = []
    for ws in (own, (both, both)):
        for _ in range(3):
            out, o = torch.full_like(q, 7.0), torch.full((2, hq, d), 7.0, device="cuda")
            sfi.sfi_prefill_attn(prompts, q, kn, kn, out, None, ws[0])
            sfi.sfi_paged_attn(lay, q[:2], k, v, o, None, ws[1])
            outs.append((out, o))
        assert sfi.sfi_read_status(ws[0]) == 0 and sfi.sfi_read_status(ws[1]) == 0
    for out, o in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(o, outs[0][1])
