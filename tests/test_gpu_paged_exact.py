"""sfi_paged_attn where the answer is known nearly to the bit: every position counts once whatever
the cuts, probabilities keep 24 bits through the tensor cores, long sums are rounded and not
truncated.  (A bound for any order of any sum grows with the length and hides all three.)"""
import numpy as np
import pytest
import torch

from tests.paged_testlib import ints
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24  # half a step of fp32, relative


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def cache(hkv, d, dtype, page, lens, seed):
    """(table, lengths, number of pages), the pages in random order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    ids, rows, at = torch.randperm(sum(need), generator=g).tolist(), [], 0
    for x in need:
        rows.append(ids[at:at + x] + [-1] * (max(need) - x))
        at += x
    return ints(rows), ints(lens), sum(need)


def run(sfi, hq, hkv, d, dtype, page, table, lens, n_pages, q, k, v):
    lay = sfi.PagedLayout(hq, hkv, d, dtype, page, n_pages, table, lens)
    ws = sfi.paged_workspace(lay)
    out, lse = torch.full((q.shape[0], hq, d), 7.0, device="cuda"), torch.full((q.shape[0], hq), 7.0, device="cuda")
    sfi.sfi_paged_attn(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    return out, lse


def rows_of(pool, table, b, g, n):
    page = pool.shape[2]
    return pool[table[b, :-(-n // page)].long(), g].reshape(-1, pool.shape[3])[:n]


@pytest.mark.parametrize("hq,hkv,d,dtype,page,lens", [
    (4, 2, 64, BF16, 16, [70000, 8191, 0, 130001]),
    (32, 8, 64, BF16, 20, [24001] * 4),
    (8, 8, 128, BF16, 64, [24576] * 12),
    (2, 2, 64, F32, 16, [90000, 40003, 90001]),
    (8, 2, 128, BF16, 16, [200000, 160001, 0, 280000]),
    (8, 8, 128, BF16, 32, [16390] * 10),
    (8, 1, 128, BF16, 5, [1, 300, 17, 4097, 16, 15]),
    (16, 1, 64, BF16, 48, [3000, 1, 129]),
    (12, 4, 128, F32, 7, [513, 8, 9, 2000, 0, 1]),
    (16, 1, 128, F32, 16, [700000]),
    (4, 4, 64, BF16, 16, [(i * 37) % 330 for i in range(500)]),
])
def test_every_position_counts_once(sfi, hq, hkv, d, dtype, page, lens):
    """With q = 0 every probability is 1, and with V of +1 and -1 every sum is a whole number below
    2^24: out is the exact sum divided by the length, and a tile lost, doubled or taken from
    elsewhere shows in nearly every one of the d sums."""
    table, n, n_pages = cache(hkv, d, dtype, page, lens, len(lens) + d)
    g = torch.Generator("cuda").manual_seed(3)
    k = torch.randn((n_pages, hkv, page, d), generator=g, device="cuda", dtype=dtype)
    v = (torch.randint(0, 2, k.shape, generator=g, device="cuda", dtype=torch.int8) * 2 - 1).to(dtype)
    q = torch.zeros(len(lens), hq, d, device="cuda", dtype=dtype)
    out, lse = run(sfi, hq, hkv, d, dtype, page, table, n, n_pages, q, k, v)
    G = hq // hkv
    for b in range(len(lens)):
        if lens[b] == 0:
            assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
            continue
        for h in range(0, hq, G):
            want = rows_of(v, table, b, h // G, lens[b]).double().sum(0)
            # (the quotient rounded once; 2 units in case of a division that is not)
            got = out[b, h:h + G].double() * lens[b]
            assert bool(((got - want).abs() <= 2 * ULP * want.abs()).all()), (b, h)
        # ln 2 log2 n: two roundings and log2f's own error of 1 ulp
        assert bool(((lse[b].double() - np.log(lens[b])).abs() <= 4 * 2 * ULP * max(1.0, np.log(lens[b]))).all()), b


def bf16(x):
    return torch.tensor(x, dtype=torch.float32).to(BF16).double().numpy()


def left_over(p, terms):
    """Of p, what `terms` bf16 terms leave, each rounding what is left (relative to p)."""
    r = np.float32(p).astype(np.float64)
    for _ in range(terms):
        r = r - bf16(r)
    return np.abs(r) / p


@pytest.mark.parametrize("G", [1, 4, 8, 11, 16])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (128, 20)])
def test_probabilities_keep_24_bits(sfi, G, d, page):
    """V = 1, so out = sum P / sum p with P the probabilities as the tensor cores get them.  In each
    tile of 16 keys one scores 0 and the others -w (exact: q and k have one element each), so p is
    1 and 2^(-c w); w is chosen so that two bf16 terms of p leave much.

    One CTA, a tile to each of its 8 warps, all with the maximum 0.  In units of 2^-24: P's sum
    over a tile 16 truncations of the sum in any order, 2 each, 7 roundings over the warps; sum p
    1 + 3 roundings in a warp and 7 over them; the quotient 1; 1 for what three terms leave and 1
    for the products of the small terms: 53."""
    bound = 53 * ULP
    grid = torch.arange(1, 2 ** 11, dtype=torch.float32).to(BF16).unique().double().numpy() / 64  # bf16 numbers up to 32
    p = np.exp(-grid / np.sqrt(d))
    worst = np.min([left_over(p * (1 + x), 2) for x in (0, 2.0 ** -22, -2.0 ** -22)], 0)  # exp2's own error
    share = 15 * p / (1 + 15 * p)
    best = np.argsort(-worst * share)[:G]
    assert (worst * share)[best].min() > 1.35 * bound and left_over(p[best], 3).max() <= ULP
    n = 128
    table, lens, n_pages = cache(1, d, BF16, page, [n], 7)
    q = torch.zeros(1, G, d, device="cuda", dtype=BF16)
    q[0, :, 3] = torch.tensor(grid[best], device="cuda").to(BF16)
    row = torch.zeros(-(-n // page) * page, d, device="cuda", dtype=BF16)
    row[:, 3] = -1
    row[5::16, 3] = 0
    k, v = (torch.zeros(n_pages, 1, page, d, device="cuda", dtype=BF16) for _ in range(2))
    k[table[0].long(), 0] = row.view(-1, page, d)
    v[:] = 1
    out, _ = run(sfi, G, 1, d, BF16, page, table, lens, n_pages, q, k, v)
    assert float((out.double() - 1).abs().max()) <= bound


def test_long_sums_are_not_truncated(sfi):
    """About a thousand tiles in a row for each warp, V positive, scores exact: a sum that truncates
    at each tile would fall behind by 0.5 2^-23 0.75 a tile of what it holds, 370 units of 2^-24
    in the end.

    Rounded sums, in units of 2^-24: T roundings, each at most one unit of what the sum holds
    then and taken as independent, come to sqrt(T) / 3 of the end, times 6 for the worst of the
    outputs, for sum p v and for sum p each; a tile's products 16 truncations in any order, 2
    each; 8 warps and up to 21 pieces joined in both sums; an error of exp2 of 4 units moves
    out by |v - out|, 0.25 on average: 1."""
    n, hq, hkv, d, page = 2_400_000, 16, 8, 64, 64
    tiles = n / 16 * hkv / torch.cuda.get_device_properties(0).multi_processor_count / 8
    bound = (2 * 6 * np.sqrt(tiles) / 3 + 32 + 2 * 29 + 4) * ULP
    assert bound < 0.6 * 0.375 * tiles * ULP
    g = torch.Generator("cuda").manual_seed(5)
    n_pages = n // page
    table, lens = torch.randperm(n_pages, generator=g, device="cuda").int()[None], ints([n])
    k = torch.randint(-1, 2, (n_pages, hkv, page, d), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    v = torch.rand(k.shape, generator=g, device="cuda", dtype=BF16) + 1
    q = torch.randint(-1, 2, (1, hq, d), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    out, lse = run(sfi, hq, hkv, d, BF16, page, table, lens, n_pages, q, k, v)
    for h in (0, 1, 6, hq - 1):
        s = rows_of(k, table, 0, h // 2, n).double() @ q[0, h].double() / d ** 0.5
        p = torch.softmax(s, 0)
        want = p @ rows_of(v, table, 0, h // 2, n).double()
        err = float(((out[0, h].double() - want) / want).abs().max())
        print("relative error", h, err, "bound", bound)
        assert err <= bound
        assert abs(float(lse[0, h]) - float(torch.logsumexp(s, 0))) <= bound + 8 * ULP * 20


@pytest.mark.parametrize("hq,hkv,d,dtype,page", [(8, 2, 128, BF16, 16), (16, 1, 64, BF16, 20), (12, 2, 64, F32, 7)])
@pytest.mark.parametrize("x", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_value_keeps_to_its_column(sfi, hq, hkv, d, dtype, page, x):
    lens = [700, 33]
    table, n, n_pages = cache(hkv, d, dtype, page, lens, 11)
    g = torch.Generator("cuda").manual_seed(7)
    k, v = (torch.randn((n_pages, hkv, page, d), generator=g, device="cuda", dtype=dtype) for _ in range(2))
    q = torch.randn(2, hq, d, generator=g, device="cuda", dtype=dtype)
    clean, lse = run(sfi, hq, hkv, d, dtype, page, table, n, n_pages, q, k, v)
    at, head, col = 345, hkv - 1, 37
    v[table[0, at // page].long(), head, at % page, col] = x
    out, lse2 = run(sfi, hq, hkv, d, dtype, page, table, n, n_pages, q, k, v)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, head * (hq // hkv):, col] = True
    assert not torch.isfinite(out[hit]).any()
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse, lse2)
