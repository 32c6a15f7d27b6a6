"""Forks of a sequence that holds a page outside the pool: flagged, the destination stays empty, no
page is taken and no count moves; the pairs beside it are served as if it were not there."""
import pytest
import torch

from tests.sfi_testlib import load_sfi
from tests.test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def spoil(p, b, i, page):
    """Sequence b's i-th page becomes `page`; returns a way back."""
    old = int(p.model.table[b, i])

    def put(x):
        p.table[b, i] = x
        p.model.table[b, i] = x
    put(page)
    return lambda: put(old)


@pytest.mark.parametrize("entry", [0, 1, 2, 40])
@pytest.mark.parametrize("bad", [-1, 1 << 24, "n"])
def test_bad_page_of_the_source(sfi, entry, bad):
    p = Pool(sfi, 2, 64, torch.bfloat16, 4, [163, 0, 6, 0, 0, 9, 0], 3, layers=2)
    back = spoil(p, 0, entry, p.lay.n_pages if bad == "n" else bad)
    sfi.sfi_pages_fork(p.lay, p.store, [2, 0, 5, 0], [1, 3, 4, 6], p.ws)
    assert p.model.fork([2, 5], [1, 4]) == set()
    p.same(["index"])
    back()
    p.fork([0, 0], [3, 6])
    p.held_counts_match()


def test_bad_last_page_of_many(sfi):
    """All pages of a batch's sources but one are fine, and the last page free goes to the last pair."""
    lens = [5] * 40 + [0] * 40
    p = Pool(sfi, 1, 64, torch.float32, 4, lens, 39, layers=1)
    back = spoil(p, 17, 1, -5)
    src, dst = list(range(40)), list(range(40, 80))
    sfi.sfi_pages_fork(p.lay, p.store, src, dst, p.ws)
    del src[17], dst[17]
    assert p.model.fork(src, dst) == set()
    p.same(["index"])
    back()
    p.held_counts_match()
    p.fork([17], [57])  # and none is left
