"""Attention for sequences that share their first pages (sfi_paged_attn_shared) against the 64-bit
restatement, and beside sfi_paged_attn."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import close, close_lse, f32_tolerance, f64, ints, normal, offsets
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


class Batch:
    """groups: (sequences, shared pages) one after another, `own` positions of each sequence behind them;
    what lies in no group shares nothing (shared pages None: sequences between groups)."""

    def __init__(self, hq, hkv, d, page, groups, own, seed=1):
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        count = [g for g, _ in groups]
        assert sum(count) == len(own)
        ids = iter(np.random.RandomState(seed).permutation(10 + sum(s or 0 for _, s in groups) + sum(-(-n // page) for n in own)).tolist())
        rows, self.lens, self.cu, self.shared, at = [], [], [], [], 0
        for m, s in groups:
            first = [next(ids) for _ in range(s or 0)]
            if s is not None:
                assert not self.cu or self.cu[-1] == at, "sequences in no group lie at the ends"
                self.cu = self.cu or [at]
                self.cu.append(at + m)
                self.shared.append(s)
            for n in own[at:at + m]:
                rows.append(first + [next(ids) for _ in range(-(-n // page))])
                self.lens.append(len(first) * page + n)
            at += m
        self.cu = self.cu or [0]
        self.n_pages = 10 + max([max(r) for r in rows if r], default=0)
        width = max(len(r) for r in rows) + 1
        self.rows = np.array([r + [-1] * (width - len(r)) for r in rows], np.int32)
        self.table, self.len = ints(self.rows.tolist()), ints(self.lens)
        self.q = normal((len(own), hq, d), BF16, seed + 1)
        self.k = normal((self.n_pages, hkv, page, d), BF16, seed + 2)
        self.v = normal((self.n_pages, hkv, page, d), BF16, seed + 3)
        self.lay = sfi_layout(self)

    def run(self, sfi, status=0, ws=None, cu=None, shared=None, plain=False):
        cu, shared = ints(self.cu if cu is None else cu), ints(self.shared if shared is None else shared)
        ws = sfi.paged_shared_workspace(self.lay, shared.numel()) if ws is None else ws
        out = torch.full((len(self.lens), self.hq, self.d), 7.0, device="cuda")
        lse = torch.full((len(self.lens), self.hq), 7.0, device="cuda")
        if plain:
            sfi.sfi_paged_attn(self.lay, self.q, self.k, self.v, out, lse, ws)
        else:
            sfi.sfi_paged_attn_shared(self.lay, cu, shared, self.q, self.k, self.v, out, lse, ws)
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == status
        return out, lse

    def check(self, out, lse, only=None):
        at = list(range(len(self.lens))) if only is None else only
        ref, rl, scale, size = P.paged(f64(self.q)[at], f64(self.k), f64(self.v), self.rows[at], [self.lens[b] for b in at])
        tol = f32_tolerance(ref, scale, size, self.d, max(self.lens), True)
        close(f64(out)[at], ref, tol, "out")
        close_lse(f64(lse)[at], rl, size, self.d)


def sfi_layout(b):
    sfi = load_sfi()
    return sfi.PagedLayout(b.hq, b.hkv, b.d, BF16, b.page, b.n_pages, b.table, b.len)


CASES = [
    # (H_q, H_kv, d, page size, [(sequences, shared pages)], own positions)
    (8, 2, 128, 16, [(2, 1)], [1, 1]),
    (8, 2, 128, 16, [(3, 8)], [5, 0, 40]),                       # a block exactly; one holds nothing of its own
    (8, 2, 64, 16, [(4, 9)], [1, 17, 300, 16]),
    (4, 4, 128, 64, [(5, 3)], [10, 20, 30, 40, 50]),             # one head a group
    (16, 1, 128, 32, [(9, 5), (2, 1)], list(range(1, 12))),      # 16 heads a group: two halves and more
    (8, 1, 64, 48, [(40, 4)], [(i * 5) % 60 for i in range(40)]),  # several tiles of a group
    (6, 2, 128, 8, [(3, 21), (4, 2)], [3, 1, 9, 70, 8, 0, 2]),   # three heads a group, boxes of 8
    (5, 1, 64, 24, [(30, 7)], [1 + i % 4 for i in range(30)]),
    (7, 1, 128, 128, [(3, 2)], [200, 1, 128]),
    (14, 2, 64, 256, [(3, 1)], [1, 2, 3]),
    (2, 1, 128, 1024, [(2, 1)], [1025, 3]),
    (8, 2, 128, 20, [(3, 13)], [5, 25, 0]),                      # gathered row by row
    (8, 2, 64, 1, [(4, 150)], [5, 2, 0, 1]),
    (3, 1, 128, 7, [(50, 40)], [1 + i % 9 for i in range(50)]),
    (12, 1, 64, 4, [(12, 70)], [1] * 12),
    # sequences of no group, groups of one, of none, and that share nothing
    (8, 2, 128, 16, [(2, None), (3, 4), (1, 6), (0, 2), (2, 0), (2, 3), (3, None)], [7, 0, 1, 2, 3, 40, 50, 60, 0, 8, 9, 100, 33]),
    (4, 1, 64, 20, [(1, None), (2, 4), (1, None)], [40, 5, 6, 0]),
    (4, 2, 64, 16, [(4, None)], [40, 5, 6, 0]),                  # no group at all
    (4, 2, 64, 16, [(1, 3)], [4]),
]


@pytest.mark.parametrize("hq,hkv,d,page,groups,own", CASES)
def test_matches_oracle(sfi, hq, hkv, d, page, groups, own):
    b = Batch(hq, hkv, d, page, groups, own)
    out, lse = b.run(sfi)
    b.check(out, lse)
    again, lse2 = b.run(sfi)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # what nobody holds may hold anything, table entries behind the held ones and the others' copies
    # of the shared ones point nowhere
    used = torch.zeros(b.n_pages, b.page, dtype=torch.bool)
    for i, n in enumerate(b.lens):
        for x in range(n):
            used[b.rows[i, x // page], x % page] = True
    for pool in (b.k, b.v):
        pool.masked_fill_(~used.cuda()[:, None, :, None], float("nan"))
    b.table[b.table < 0] = 1 << 30
    for (m, s), at in zip([g for g in groups if g[1] is not None], b.cu):
        if m > 1:
            b.table[at + 1:at + m, :s] = -9
    again, lse2 = b.run(sfi)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq,hkv,d,page,groups,hi", [
    (32, 8, 128, 64, [(64, 80)], 300),               # two halves, shares of several blocks
    (8, 8, 64, 16, [(130, 40), (3, 260)], 90),       # more than 128 sequences of one head
    (32, 2, 128, 16, [(33, 130), (20, 64), (2, 500)], 200),
    (16, 4, 128, 40, [(9, 100), (8, 101), (40, 30)], 400),
    (8, 2, 64, 12, [(20, 700)], 100),
    (4, 1, 128, 256, [(3, 200)], 3000),
])
def test_long_prefixes_are_cut_and_joined(sfi, hq, hkv, d, page, groups, hi):
    n = sum(m for m, _ in groups)
    b = Batch(hq, hkv, d, page, groups, [(i * 37) % hi for i in range(n)], seed=5)
    out, lse = b.run(sfi)
    again, lse2 = b.run(sfi)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    b.check(out, lse, only=sorted({0, 1, b.cu[1] - 1, b.cu[-2], n // 2, n - 1}))


@pytest.mark.parametrize("page", [16, 12, 20])
def test_shares_that_hold_several_pieces(sfi, page):
    """More units than SMs, of several blocks each, in one half and in two: a CTA goes from one to the next."""
    b = Batch(32, 8, 128, page, [(m, 1 + (7 * m + i) % 19) for i, m in enumerate([2, 9, 40, 3, 33, 64, 5, 2, 70, 8] * 2)],
              [(i * 5) % 23 for i in range(472)])
    out, lse = b.run(sfi)
    for _ in range(8):
        again, lse2 = b.run(sfi)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    b.check(out, lse, only=list(range(0, 472, 29)) + [471])


@pytest.mark.parametrize("page", [16, 12])
def test_many_groups(sfi, page):
    """As many groups as a batch may have, each of two sequences: more tiles than SMs."""
    b = Batch(2, 2, 64, page, [(2, 1 + i % 3) for i in range(512)], [1 + i % 5 for i in range(1024)])
    b.check(*b.run(sfi))


@pytest.mark.parametrize("end", [0.1, 6.0])
def test_growing_scores_rescale(sfi, end):
    """Scores that grow, or fall, along the prefix and the own positions."""
    b = Batch(4, 1, 128, 16, [(3, 90)], [100, 7, 33])
    ramp = torch.linspace(6.1 - end, end, 90, device="cuda")
    b.k[b.rows[0, :90].tolist()] *= ramp[:, None, None, None].to(BF16)
    b.check(*b.run(sfi))


def test_scores_of_different_sequences(sfi):
    """Queries from 2^-8 to 2^6 in one tile, one of zeros: each row has its own maximum."""
    b = Batch(4, 1, 64, 16, [(6, 40)], [3, 0, 50, 1, 20, 9])
    b.q *= torch.exp2(torch.tensor([-8.0, 6.0, 0.0, 3.0, -2.0, 0.0], device="cuda")).to(BF16)[:, None, None]
    b.q[5] = 0
    b.check(*b.run(sfi))


def test_query_that_is_not_finite_stays_alone(sfi):
    b = Batch(8, 2, 64, 16, [(6, 20)], [3, 0, 50, 1, 20, 9])
    good, gl = b.run(sfi)
    b.q[2, 5, 7] = float("nan")
    out, lse = b.run(sfi)
    assert out[2, 5].isnan().all() and lse[2, 5].isnan()
    rest = torch.ones(6, 8, dtype=torch.bool, device="cuda")
    rest[2, 5] = False
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], gl[rest])


@pytest.mark.parametrize("page,own", [(16, [5, 0, 40]), (12, [300, 1, 9])])
def test_what_is_not_finite_reaches_the_group(sfi, page, own):
    """Keys of NaN over whole blocks, so that a state holds nothing else; and an element of V that is
    not finite at a position whose probability is 0 in fp32."""
    pages = 288 // page  # six blocks of 48, each a share by itself
    b = Batch(8, 2, 128, page, [(3, pages), (2, pages)], own + [7, 8])
    good, gl = b.run(sfi)
    rest = torch.ones(5, 8, dtype=torch.bool, device="cuda")
    rest[:3, 4:] = False
    held = b.rows[0, :96 // page].tolist()
    keep = b.k[held, 1].clone()
    b.k[held, 1] = float("nan")
    out, lse = b.run(sfi)
    assert out[:3, 4:].isnan().all() and lse[:3, 4:].isnan().all()
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], gl[rest])
    b.k[held, 1] = keep
    # sequence 0's heads 4 to 7 ask for what those keys are not: scores of about -200 and less
    b.q[0, 4:] = b.q[0, 4:].abs()
    b.k[held, 1] = -25.0
    b.v[held[0], 1, 3, 17] = float("nan")
    out, lse = b.run(sfi)
    bad = out[0, 4:].isnan()
    assert bad[:, 17].all() and int(bad.sum()) == 4 and torch.isfinite(lse).all()
    assert torch.equal(out[rest], good[rest])


def test_wrong_groups_share_nothing(sfi):
    """Flagged, and every sequence is attended to by its own row of the table."""
    b = Batch(8, 2, 128, 16, [(3, 4), (2, 3)], [5, 0, 40, 1, 9])
    alone, al = b.run(sfi, shared=[0, 0])
    b.check(alone, al)
    for cu in ([0, 4, 3], [-1, 3, 5], [0, 3, 6], [3, 0, 5], [0, 3, 1 << 30], [0, -(1 << 31), 5]):
        out, lse = b.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP, cu=cu)
        assert torch.equal(out, alone) and torch.equal(lse, al), cu
    # the second group only
    for shared in ([4, 4], [4, -1], [4, 1000], [4, 1 << 30]):
        out, lse = b.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP, shared=shared)
        b.check(out, lse)
    for n in (-5, 1 << 20):
        b.len[4] = n
        out, lse = b.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP | (sfi.SFI_DEV_BAD_INDEX if n > 0 else 0))
        b.check(out, lse, only=[0, 1, 2, 3])
        assert n > 0 or (out[4] == 0).all()


def test_bad_page_is_flagged(sfi):
    b = Batch(8, 2, 128, 16, [(3, 4), (2, 3)], [5, 0, 40, 1, 9])
    good, _ = b.run(sfi)
    for page in (b.n_pages, -1, 1 << 30):
        b.table[0, 2] = page
        out, _ = b.run(sfi, status=sfi.SFI_DEV_BAD_INDEX)
        assert torch.equal(out[3:], good[3:])


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 2, 64, 32), (8, 2, 128, 20)])
def test_wait_limit(sfi, hq, hkv, d, page):
    """A one-clock limit: the waits give up, the status says so, nothing is left in flight; afterwards
    the default limit gives the bytes from before."""
    b = Batch(hq, hkv, d, page, [(40, 16000 // page), (3, 4000 // page)], [(i * 37) % 200 for i in range(43)])
    good, _ = b.run(sfi)
    ws = sfi.paged_shared_workspace(b.lay)
    cu, shared, out = ints(b.cu), ints(b.shared), torch.empty_like(good)
    sfi.lib.sfi_set_wait_limit(1)
    try:
        for _ in range(2):
            sfi.sfi_paged_attn_shared(b.lay, cu, shared, b.q, b.k, b.v, out, None, ws)
            assert sfi.sfi_read_status(ws) == sfi.SFI_DEV_WAIT_TIMEOUT
    finally:
        sfi.lib.sfi_set_wait_limit(0)
    ws.zero_()
    again, _ = b.run(sfi, ws=ws)
    assert torch.equal(good, again)


def test_workspace_serves_the_other_calls(sfi):
    """Shared, paged and prompt attention in turn on one workspace, fewer groups than it is for."""
    b = Batch(8, 2, 128, 16, [(3, 4), (2, 3)], [5, 0, 40, 1, 9])
    ws = sfi.paged_shared_workspace(b.lay)
    first = b.run(sfi, ws=ws)
    plain = b.run(sfi, ws=ws, plain=True)
    one = b.run(sfi, ws=ws, cu=[0, 3], shared=[4])
    packed = sfi.PackedLayout(8, 2, 128, BF16, ints([0, 50]), ints([0, 50]), 50, 50)
    q, k, v = normal((50, 8, 128), BF16, 1), normal((50, 2, 128), BF16, 2), normal((50, 2, 128), BF16, 3)
    sfi.sfi_prefill_attn(packed, q, k, v, torch.empty_like(q), None, ws)
    again = b.run(sfi, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    for out, lse in (plain, one):
        b.check(out, lse)
    none = b.run(sfi, ws=ws, cu=[0], shared=[])
    assert torch.equal(none[0], plain[0])


def test_empty_groups(sfi):
    """1024 groups, of which two have sequences.  Some of the others name more pages than a row of
    the table has, which is flagged and changes nothing."""
    b = Batch(8, 2, 64, 16, [(3, 4), (2, 3)], [5, 0, 40, 1, 9])
    good = b.run(sfi)
    cu = [0] * 500 + [3] * 300 + [5] * 225
    shared = [7 * (i % 5) for i in range(1024)]
    shared[499], shared[799] = 4, 3
    assert max(shared) > b.rows.shape[1]
    out, lse = b.run(sfi, status=sfi.SFI_DEV_LEN_OVER_CAP, cu=cu, shared=shared)
    assert torch.equal(out, good[0]) and torch.equal(lse, good[1])


def test_graphs_on_one_workspace(sfi):
    """Two captured calls of different groups and an eager one, in turn on one workspace and on a
    stream of the caller's; a replay reads the groups and lengths of its time."""
    b, c = Batch(8, 2, 128, 16, [(3, 4), (2, 3)], [5, 0, 40, 1, 9]), Batch(8, 2, 128, 20, [(2, 9), (3, 30)], [50, 7, 40, 1, 0], seed=3)
    sizes = [sfi.paged_shared_workspace(x.lay).numel() for x in (b, c)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    want = [b.run(sfi), c.run(sfi)]
    args, outs, graphs = [], [], []
    for x in (b, c):
        args.append((x.lay, ints(x.cu), ints(x.shared), x.q, x.k, x.v))
        outs.append((torch.zeros(5, 8, 128, device="cuda"), torch.zeros(5, 8, device="cuda")))
        sfi.sfi_paged_attn_shared(*args[-1], *outs[-1], ws)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sfi.sfi_paged_attn_shared(*args[-1], *outs[-1], ws)
    eager = tuple(torch.zeros_like(t) for t in outs[0])
    st = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            for t in o:
                t.zero_()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for g in graphs:
                g.replay()
            sfi.sfi_paged_attn_shared(*args[0], *eager, ws)
        st.synchronize()
        for got, good in zip(outs + [eager], want + want[:1]):
            assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    args[0][2].copy_(ints([2, 0]))  # fewer pages, and a group that shares nothing
    b.len[0] -= 3
    b.lens[0] -= 3
    graphs[0].replay()
    torch.cuda.synchronize()
    b.check(*outs[0])
    assert sfi.sfi_read_status(ws) == 0


def test_forked_sequences_decode(sfi):
    """A prompt, forked; every sequence appends tokens, some of them captured in a graph: the group attends
    as each by itself does."""
    hq, hkv, d, page, B = 8, 2, 128, 16, 6
    table = torch.full((B, 20), -1, dtype=torch.int32, device="cuda")
    ln = torch.zeros(B, dtype=torch.int32, device="cuda")
    lay = sfi.PagedLayout(hq, hkv, d, BF16, page, 60, table, ln)
    k, v = (torch.full((60, hkv, page, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    store = sfi.PageStore(torch.zeros(60, dtype=torch.int32, device="cuda"), k, v)
    ws = sfi.paged_shared_workspace(lay, 2)
    n = 200
    sfi.sfi_pages_extend(lay, store, ints([n, 0, 0, 0, 70, 0]), ws)
    new = [normal((n + 70, hkv, d), BF16, 30 + i) for i in range(2)]
    sfi.sfi_paged_append(lay, *new, k, v, ints([0, n, n, n, n, n + 70, n + 70]), ws)
    sfi.sfi_pages_fork(lay, store, [0, 0, 0, 4], [1, 2, 3, 5], ws)
    cu, shared = ints([0, 4, 6]), ints([n // page, 70 // page])
    q, kn, vn = normal((B, hq, d), BF16, 40), normal((B, hkv, d), BF16, 41), normal((B, hkv, d), BF16, 42)
    out, lse, out2, lse2 = torch.empty(B, hq, d, device="cuda"), torch.empty(B, hq, device="cuda"), torch.empty(B, hq, d, device="cuda"), torch.empty(B, hq, device="cuda")

    def step():
        sfi.sfi_pages_extend(lay, store, None, ws)
        sfi.sfi_paged_append(lay, kn, vn, k, v, None, ws)
        sfi.sfi_paged_attn_shared(lay, cu, shared, q, k, v, out, lse, ws)

    def check():
        torch.cuda.synchronize()
        assert sfi.sfi_read_status(ws) == 0
        rows = table.cpu().numpy()
        kk, vv = (np.nan_to_num(f64(x)) for x in (k, v))
        ref, rl, scale, size = P.paged(f64(q), kk, vv, rows, ln.tolist())
        sfi.sfi_paged_attn(lay, q, k, v, out2, lse2, ws)
        for o, z in ((out, lse), (out2, lse2)):
            close(f64(o), ref, f32_tolerance(ref, scale, size, d, 300, True), "out")
            close_lse(f64(z), rl, size, d)

    step()
    check()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(20):
        for x, s in ((q, 50), (kn, 80), (vn, 110)):
            x.copy_(normal(x.shape, BF16, s + i))
        graph.replay()
        if i % 6 == 0:
            check()
    check()
    # the second group ends; the first shares less than it could; on a stream of its own
    sfi.sfi_pages_free(lay, store, [4, 5], ws)
    shared.copy_(ints([3, 0]))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    sfi.sfi_paged_attn_shared(lay, cu, shared, q, k, v, out, lse, ws, stream=st)
    st.synchronize()
    check()
    assert (out[4:] == 0).all()


def test_pool_beyond_2_31_elements(sfi):
    """Shared pages far behind the pool's start, by boxes and gathered."""
    for page in (16, 12):
        b = Batch(4, 1, 64, page, [(3, 11)], [5, 0, 40])
        apart = 1 << 27  # elements between pages
        far = torch.zeros((b.n_pages - 1) * apart + b.k[0].numel(), dtype=BF16, device="cuda")
        pools = []
        for x in (b.k, b.v):
            pools.append(far.as_strided((b.n_pages, 1, page, 64), (apart, page * 64, 64, 1), len(pools) * 65536) if not pools else None)
            if pools[-1] is None:
                pools[-1] = far[:-65536].as_strided((b.n_pages - 1, 1, page, 64), (apart, page * 64, 64, 1), 65536)
        # (K in pages 0 .., V 65536 elements behind each; the last page is left to K)
        n = b.n_pages - 1
        assert b.rows.max() < n
        kp, vp = pools[0][:n], pools[1]
        kp.copy_(b.k[:n])
        vp.copy_(b.v[:n])
        lay = sfi.PagedLayout(4, 1, 64, BF16, page, n, b.table, b.len, page_stride=apart)
        assert n * apart > 1 << 31
        ws = sfi.paged_shared_workspace(lay, 1)
        out, lse = torch.empty(3, 4, 64, device="cuda"), torch.empty(3, 4, device="cuda")
        sfi.sfi_paged_attn_shared(lay, ints(b.cu), ints(b.shared), b.q, kp, vp, out, lse, ws)
        assert sfi.sfi_read_status(ws) == 0
        b.check(out, lse)
        del far, pools, kp, vp
        torch.cuda.empty_cache()


def test_binding_refusals(sfi):
    b = Batch(8, 2, 128, 16, [(3, 4)], [5, 0, 40])
    ws = sfi.paged_shared_workspace(b.lay, 1)
    out = torch.empty(3, 8, 128, device="cuda")
    ok = dict(cu_group=ints(b.cu), shared_pages=ints(b.shared), q=b.q, k=b.k, v=b.v, out=out, ws=ws)
    for bad in (dict(cu_group=ints([0])), dict(cu_group=ints(b.cu).long()), dict(shared_pages=ints([1, 2])), dict(q=b.q[:2]),
                dict(out=out.bfloat16()), dict(k=b.k[:1]), dict(cu_group=ints(b.cu, "cpu"))):
        with pytest.raises(ValueError):
            sfi.sfi_paged_attn_shared(b.lay, **{**ok, **bad})
    with pytest.raises(sfi.SfiError):
        sfi.sfi_paged_attn_shared(b.lay, **{**ok, "ws": sfi.paged_workspace(b.lay)})
