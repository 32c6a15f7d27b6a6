"""Units of many pieces, and probabilities of many bits: attention over an 8-bit cache and over shared
prefixes where values do not average out, within bounds that a lost or exchanged piece, or a
dropped term of the probabilities, leaves (which the CPU tests show)."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import close, close_lse, f64, ints, pool_of, score_error
from tests.sfi_testlib import load_sfi
from tests.test_gpu_shared import Batch

gpu = pytest.mark.gpu
BF16, F32, I8, E4M3 = torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn
SHARES = 152  # that the line of tiles is cut into, at most


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def rows_of(n, hkv, d, seed):
    """K and V [hkv, n, d] of one sequence: noise, and along the positions scores that grow by about 2 (for queries
    around 1) and values that grow from 1 to 2."""
    g = torch.Generator().manual_seed(seed)
    at = torch.linspace(0, 1, n)[None, :, None]
    return (0.25 * torch.randn(hkv, n, d, generator=g) + (at - 0.5) * (2 / d ** 0.5),
            1 + at + 0.25 * torch.randn(hkv, n, d, generator=g))


def queries(shape, dtype, seed, device="cuda"):
    return (1 + 0.5 * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(device)


def bound(ref, scale, size, d, adds, extra=0.0):
    """Elementwise: scores off as in the other tests, exp2 by 2^-22 twice, and a sum of `adds` fp32 additions one
    after another (a truncation in a tensor core counts as two), half a step of the sum of
    magnitudes each, in the numerator and in the sum of the probabilities."""
    move = np.expm1(2 * score_error(size, d))[..., None] + 2.0 ** -21 + 2 * adds * 2.0 ** -24 + extra
    return move * (scale + np.abs(ref))


def adds_q8(n):
    """A warp's lane adds at most n / 8 / 32 tiles to its sums, four probabilities of each to l; a tile's
    products start from zero, 64 products with their two terms in 8 truncations; 8 warps and
    as many pieces as shares are joined."""
    return 16 + n // 64 + 4 + 5 + 8 + SHARES + 16


def adds_shared(n0, own, all_own):
    """Four blocks of 48 keys in tensor memory, 18 truncations a block; then an addition for four
    blocks, and for l one for a block; the pieces, at most as many as shares, and 8 warps.  Own
    positions in tiles of 16 (two truncations each, or two probabilities of a lane), of which `all_own`
    positions of all sequences and KV heads give each of 8 warps on each SM its piece; those are joined."""
    tiles = -(-all_own // 16 // (8 * SHARES)) + 1
    return 2 * 4 * 18 + n0 // 48 + 16 + SHARES + 8 + 4 * tiles + own // 16 // max(1, tiles - 1) + 2


# ------------------------------------------------------------------- what the bounds see

@pytest.mark.parametrize("n,d,adds", [(280000, 128, adds_q8(280000)), (70000, 64, adds_q8(70000)), (90001, 128, adds_q8(90001)),
                                      (51200, 128, adds_shared(51200, 0, 0)), (20000, 64, adds_shared(48, 20000, 60000))])
def test_a_lost_piece_leaves_the_bound(n, d, adds):
    """Lost, counted twice, or with another piece's values: nearly every element is out of bounds."""
    K, V = (x[0].double().numpy() for x in rows_of(n, 1, d, 3))
    q = f64(queries((d,), BF16, 4, "cpu"))
    ref, _, scale, size = P.attend(q, K, V, n)
    tol = bound(ref[None], scale[None], np.array([size]), d, adds)[0]
    s = K @ q / np.sqrt(d)
    p = np.exp(s - s.max())
    p /= p.sum()
    step = n // SHARES
    parts = [slice(i * step, (i + 1) * step) for i in (0, SHARES // 2, SHARES - 1)]
    for at in parts:
        lost = p[at] @ V[at]
        assert (np.abs(lost) > tol).mean() > 0.9, (at, lost.min(), tol.max())
    a, b = parts[0], parts[2]
    assert (np.abs(p[a] @ V[b] + p[b] @ V[a] - p[a] @ V[a] - p[b] @ V[b]) > tol).mean() > 0.9
    assert (np.abs(ref) > 50 * tol).all()


def hard_score(d):
    """A score (of q = (1, 2^-8, 0, ..) and two bf16 elements of k) whose probability 2^(c s), c = log2(e) / sqrt(d),
    has most of what three bf16 terms hold and two do not, some units in the last place up or down."""
    c = np.float32(1.4426950408889634 / np.sqrt(d))
    for i in range(64, 1, -1):
        for j in range(-127, 128):
            a, b = -i / 32 * d ** 0.5 / 2, j / 32.0
            a = float(torch.tensor(a).to(BF16))
            s = np.float32(a + b * 2.0 ** -8)
            p = np.exp2(np.float64(np.float32(s * c)))
            if not 0.25 < p < 1:
                continue
            off = [1 - two_terms(np.float32(p) * (1 + u * 2.0 ** -23)) for u in range(-8, 9)]
            if min(off) > 2.0 ** -16.2:
                return a, b, p
    raise AssertionError("no such score")


def two_terms(p):
    """Share of p that its two upper terms of 8 bits hold."""
    left = np.float64(np.float32(p))
    for _ in range(2):
        e = 2.0 ** (np.floor(np.log2(left)) - 7) if left > 0 else 1.0
        left -= np.floor(left / e) * e
    return 1 - left / np.float64(np.float32(p))


TERMS = 2.0 ** -18


@pytest.mark.parametrize("d", [64, 128])
def test_two_terms_leave_the_bound(d):
    """One key of probability 1 and 47 of the hard one, values of 1: with two terms the output is out of
    bounds; with three, 24 bits, nothing is lost."""
    _, _, p = hard_score(d)
    assert 1 - (1 + 47 * p * two_terms(p)) / (1 + 47 * p) > 2 * TERMS


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,members", [(4, 3), (8, 40)])
def test_probabilities_are_not_rounded(sfi, d, hq, members):
    """The keys of the CPU test in a block of shared positions.  The bound: 18 truncations of 2^-23 in
    the tensor cores, 12 additions to the sum of the probabilities and 8 roundings of the join and of
    the division, 2^-24 each: 3.3e-6 < 2^-18.  (An error of exp2 is the same in both sums.)"""
    a, b, _ = hard_score(d)
    x = Batch(hq, 1, d, 48, [(members, 1)], [0] * members)
    x.q.zero_()
    x.q[..., 0], x.q[..., 1] = 1.0, 2.0 ** -8
    x.k.zero_()
    x.k[x.rows[0, 0], 0, 1:, 0], x.k[x.rows[0, 0], 0, 1:, 1] = a, b
    x.v.fill_(1.0)
    out, _ = x.run(sfi)
    assert float((out.double() - 1).abs().max()) < TERMS


# ------------------------------------------------------------------- long units

@gpu
@pytest.mark.parametrize("hq,hkv,d,fmt,dtype,page,lens", [
    (4, 1, 64, I8, BF16, 16, [70000, 8191, 0, 130001]), (16, 1, 128, I8, F32, 20, [90001]), (32, 8, 64, E4M3, BF16, 64, [24001] * 4),
    (8, 2, 128, E4M3, BF16, 16, [200000, 280000]),
])
def test_long_units_of_8_bit_rows(sfi, hq, hkv, d, fmt, dtype, page, lens):
    n_pages, rows = pool_of(lens, page, 3, 60)
    lay = sfi.PagedLayout(hq, hkv, d, fmt, page, n_pages, ints(rows.tolist()), ints(lens))
    k, v = (torch.zeros(n_pages, lay.page_bytes, dtype=torch.uint8, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        if n == 0:
            continue
        count = -(-n // page)
        ids = torch.from_numpy(rows[b][:count]).long().cuda()
        for pool, x in zip((k, v), rows_of(n, hkv, d, 70 + b)):
            x = torch.nn.functional.pad(x.cuda(), (0, 0, 0, count * page - n)).view(hkv, count, page, d).transpose(0, 1)
            scale = x.abs().amax(-1) / (127 if fmt == I8 else 448) + 1e-30
            lay.scales(pool)[ids] = scale
            lay.codes(pool).view(torch.uint8)[ids] = (x / scale[..., None]).round().to(fmt).view(torch.uint8) if fmt == I8 else \
                (x / scale[..., None]).to(fmt).view(torch.uint8)
    q = queries((len(lens), hq, d), dtype, 62)
    out, lse = torch.empty(len(lens), hq, d, device="cuda"), torch.empty(len(lens), hq, device="cuda")
    ws = sfi.paged_workspace(lay)
    sfi.sfi_paged_attn_q8(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    for b, n in enumerate(lens):
        if n == 0 or b not in (0, len(lens) - 1):
            continue
        ids = rows[b][:-(-n // page)].tolist()
        for h in sorted({0, hkv - 1}):
            K, V = ((f64(lay.codes(x)[:, h].view(torch.uint8)[ids].view(fmt).float()) * f64(lay.scales(x)[ids, h])[..., None]).reshape(-1, d)[:n]
                    for x in (k, v))
            for e in sorted({0, hq // hkv - 1}):
                head = h * (hq // hkv) + e
                ref, rl, scale, size = P.attend(f64(q[b, head]), K, V, n)
                # (three factors of a score; fp32 queries in 22 bits; p in 22 bits, what is below 2^-39 of the largest
                # p sv of a tile dropped: far less than 2^-24 of a sum where all weigh about the same)
                size = np.array([size * (1 + (2.0 ** -21 if dtype == F32 else 0) / (2.0 ** -23 * d))])
                close(f64(out[b, head])[None], ref[None], bound(ref[None], scale[None], size, d + 8, adds_q8(n), 2.0 ** -22 + 2.0 ** -24), "out")
                close_lse(f64(lse[b, head])[None], np.array([rl]), size, d + 8)


@gpu
@pytest.mark.parametrize("hq,hkv,d,page,members,shared,own", [
    (4, 1, 128, 256, 3, 200, 1000),     # a prefix of 51200 in as many pieces as there are SMs
    (8, 1, 64, 20, 40, 900, 30),        # both halves of a tile, and a second tile; gathered row by row
    (16, 2, 128, 16, 20, 500, 100),
    (4, 1, 64, 16, 3, 3, 20000),        # own positions in many pieces
])
def test_long_shared_prefixes(sfi, hq, hkv, d, page, members, shared, own):
    lens = [max(1, own - 7 * i % 50) for i in range(members)]
    b = Batch(hq, hkv, d, page, [(members, shared)], lens, seed=6)
    n0 = shared * page
    b.q = queries(b.q.shape, BF16, 8)
    for seq in range(members):
        first = 0 if seq == 0 else n0  # (the shared rows are the first sequence's)
        rows = rows_of(b.lens[0] if seq == 0 else b.lens[seq], hkv, d, 80 + seq)
        at = torch.arange(first, b.lens[seq])
        ids = torch.from_numpy(b.rows[seq]).long()[at // page].cuda()
        for pool, x in zip((b.k, b.v), rows):
            pool[ids, :, (at % page).cuda()] = x[:, first:].transpose(0, 1).to(BF16).cuda()
    out, lse = b.run(sfi)
    for seq in sorted({0, members // 2, members - 1}):
        ref, rl, scale, size = P.paged(f64(b.q)[[seq]], f64(b.k), f64(b.v), b.rows[[seq]], [b.lens[seq]])
        close(f64(out)[[seq]], ref, bound(ref, scale, size, d, adds_shared(n0, b.lens[seq] - n0, hkv * (sum(b.lens) - members * n0))), "out")
        close_lse(f64(lse)[[seq]], rl, size, d)
