"""Offsets of new rows that do not all ascend: the pairs that are in order are stored, every row of
them, whatever stands between; the others are flagged and left out."""
import random

import pytest
import torch

from tests.paged_testlib import f64, ints, normal
from tests.sfi_testlib import load_sfi
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def in_order(cu, lens, total):
    return [0 <= a <= b <= total and b - a <= n for a, b, n in zip(cu, cu[1:], lens)]


def store_and_check(sfi, cu, lens, total, page=4, hkv=2, d=64, seed=5):
    p = Pool(sfi, hkv, d, BF16, page, lens, 1)
    kn, vn = normal((total, hkv, d), BF16, seed), normal((total, hkv, d), BF16, seed + 1)
    sfi.sfi_paged_append(p.lay, kn, vn, p.k[1], p.v[1], ints(cu), p.ws)
    good = in_order(cu, lens, total)
    for b, ok in enumerate(good):
        if ok:
            m = cu[b + 1] - cu[b]
            p.model.append(1, f64(kn)[cu[b]:cu[b + 1]], f64(vn)[cu[b]:cu[b + 1]], [0] * (b + 1) + [m] * (len(lens) - b))
    p.same([] if all(good) else ["len"])


@pytest.mark.parametrize("cu,lens,total", [
    ([0, 100, 4, 8], [9, 9, 9], 10),              # the first leaves the rows, the second descends
    ([0, 6, 2, 8], [9, 9, 9], 8),                 # two that are in order hold the same rows
    ([5, 3, 9, -1, 4, 4, 10], [9] * 6, 10),
    ([0, 9, 5, 9], [8, 9, 9], 9),                 # the first has more rows than positions
    ([2, 2, 2, 7, 7, 7], [0, 3, 6, 0, 5], 10),    # empty ones, rows before and behind all
    ([7, 0], [9], 9),
])
def test_pairs_in_order_are_stored(sfi, cu, lens, total):
    store_and_check(sfi, cu, lens, total)


@pytest.mark.parametrize("batch", [33, 300, 1024])
def test_many_pairs(sfi, batch):
    """A sequence in ten has a bad pair, and most of the others hold nothing to a few rows."""
    r = random.Random(batch)
    cu, at = [0], 0
    for b in range(batch):
        at += r.choice([0, 0, 1, 1, 2, 5])
        cu.append(at)
    total = at
    lens = [r.randint(5, 12) for _ in range(batch)]
    store_and_check(sfi, cu, lens, total, page=8)
    for b in r.sample(range(1, batch), batch // 10):
        cu[b] = r.choice([-3, total + 1, cu[b] + r.randint(1, 40), max(0, cu[b] - r.randint(1, 40))])
    store_and_check(sfi, cu, lens, total, page=8)
