"""Attention for sequences that share their first pages (sfi_paged_attn_shared): what the softmax leaves
out weighs nothing, as in sfi_paged_attn; and what is flagged."""
import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import close, close_lse, f32_tolerance, f64
from tests.sfi_testlib import load_sfi
from tests.test_gpu_shared import Batch

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def leave_out(b, seq, positions, value):
    """Positions of sequence `seq` whose scores lie some 200 below its others' (the queries are
    positive), with `value` in V."""
    if not hasattr(b, "left"):
        b.left, b.q = torch.zeros(b.n_pages, b.page, dtype=torch.bool, device="cuda"), b.q.abs()
    for x in positions:
        at = int(b.rows[seq, x // b.page]), slice(None), x % b.page
        b.k[at] = -25.0
        b.v[at] = value
        b.left[at[0], at[2]] = True


def check_kept(b, out, lse):
    """Against the 64-bit restatement; the bound's size of scores is that of the positions that
    count (a probability of 0 is 0 with its score's error too)."""
    ref, rl, scale, _ = P.paged(f64(b.q), f64(b.k), f64(b.v), b.rows, b.lens)
    kept = b.k.masked_fill(b.left[:, None, :, None], 0.0)
    size = P.paged(f64(b.q), f64(kept), f64(b.v), b.rows, b.lens)[3]
    close(f64(out), ref, f32_tolerance(ref, scale, size, b.d, max(b.lens), True), "out")
    close_lse(f64(lse), rl, size, b.d)


@gpu
@pytest.mark.parametrize("value", [5e35, -5e35, 1e31])
@pytest.mark.parametrize("hq,hkv,d,page,members,shared,own", [
    (8, 2, 128, 16, 3, 18, [5, 0, 40]),      # six blocks of 48 keys, a share each
    (8, 2, 64, 12, 3, 24, [300, 1, 9]),      # gathered row by row; own positions in several pieces
    (8, 1, 128, 48, 40, 30, [3, 70]),        # both halves of a tile, and a second tile
])
def test_large_values_that_the_softmax_leaves_out(sfi, value, hq, hkv, d, page, members, shared, own):
    """Finite values of any size weigh nothing where the weight is 0 in fp32, as in sfi_paged_attn:
    in whole blocks of the shared part, in every other one, and in all of a sequence's own part."""
    n = shared * page
    b = Batch(hq, hkv, d, page, [(members, shared)], [own[i % len(own)] for i in range(members)], seed=3)
    leave_out(b, 0, range(48, 144), value)
    leave_out(b, 0, [x for x in range(192, n) if x // 48 % 2], value)
    for seq in range(0, members, 2):
        leave_out(b, seq, range(n, b.lens[seq]), value)
    check_kept(b, *b.run(sfi, plain=True))
    check_kept(b, *b.run(sfi))


@gpu
@pytest.mark.parametrize("page", [16, 12])
def test_large_values_of_a_whole_prefix(sfi, page):
    """The shared part as a whole is left out, and the own one decides; and the other way round."""
    b = Batch(8, 2, 128, page, [(3, 288 // page)], [60, 7, 1], seed=4)
    k, v = b.k.clone(), b.v.clone()
    leave_out(b, 0, range(288), 1e36)
    check_kept(b, *b.run(sfi))
    b.k, b.v = k, v
    b.left[:] = False
    for seq in range(3):
        leave_out(b, seq, range(288, b.lens[seq]), 1e36)
    check_kept(b, *b.run(sfi))


@gpu
def test_groups_of_a_batch_of_one(sfi):
    """Nothing can be shared, but what the groups say is looked at all the same."""
    b = Batch(8, 2, 128, 16, [(1, 4)], [9])
    good = b.run(sfi)
    b.check(*good)
    for cu, shared, status in (([0, 1], [4], 0), ([0, 0], [4], 0), ([1, 1], [4], 0), ([0, 1], [0], 0),
                               ([0, 2], [4], sfi.SFI_DEV_LEN_OVER_CAP), ([-1, 1], [4], sfi.SFI_DEV_LEN_OVER_CAP),
                               ([1, 0], [4], sfi.SFI_DEV_LEN_OVER_CAP), ([0, 1, 0], [4, 0], sfi.SFI_DEV_LEN_OVER_CAP),
                               ([0, 1], [-1], sfi.SFI_DEV_LEN_OVER_CAP), ([0, 1], [1000], sfi.SFI_DEV_LEN_OVER_CAP),
                               ([0, 1], [5], sfi.SFI_DEV_LEN_OVER_CAP)):
        out, lse = b.run(sfi, status=status, cu=cu, shared=shared)
        assert torch.equal(out, good[0]) and torch.equal(lse, good[1]), (cu, shared)
    none = b.run(sfi, cu=[0], shared=[])
    assert torch.equal(none[0], good[0]) and torch.equal(none[1], good[1])
