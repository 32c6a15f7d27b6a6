"""How far a V row that is not finite reaches inside its own sequence (sfi_prefill_attn): the rows
that attend to it, and at most 126 + 128 // G positions before it."""
import pytest
import torch

from tests.paged_testlib import ints, normal
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def run(sfi, q, k, v):
    n, m = q.shape[0], k.shape[0]
    lay = sfi.PackedLayout(q.shape[1], k.shape[1], q.shape[2], BF16, ints([0, n]), ints([0, m]), n, m)
    ws = sfi.prefill_workspace(lay)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    sfi.sfi_prefill_attn(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 16])
@pytest.mark.parametrize("context,rows", [(0, 700), (3, 560), (129, 650), (2000, 300)])
def test_reach_of_a_non_finite_value(sfi, d, G, context, rows):
    keys = context + rows
    q, k = normal((rows, G, d), BF16, 1), normal((keys, 1, d), BF16, 2)
    v = normal((keys, 1, d), BF16, 3)
    clean, lse = run(sfi, q, k, v)
    for at in (255, 256, 300, keys - 130, keys - 1):
        for x in (float("nan"), float("inf")):
            w = v.clone()
            w[at] = x
            out, lse2 = run(sfi, q, k, w)
            assert torch.equal(lse, lse2)
            far = max(0, at - (126 + 128 // G) - context)  # rows before this one keep their bits
            assert torch.equal(out[:far], clean[:far])
            assert not torch.isfinite(out[max(0, at - context):].float()).any()
            # a row between is either spoilt or as it was
            near, same = out[far:max(0, at - context)], clean[far:max(0, at - context)]
            assert bool((~torch.isfinite(near.float()) | (near == same)).all())
