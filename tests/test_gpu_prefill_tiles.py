"""Prompt attention where a CTA takes tile after tile: packed prompts of all lengths, so that tiles
with two halves and with one, last key blocks that end inside and at a block, and sequences with and
without context follow each other in every CTA."""
import random

import pytest
import torch

import oracle.paged_oracle as P
from tests.paged_testlib import bf16_tolerance, close, close_lse, f64, ints, normal, offsets
from tests.sfi_testlib import load_sfi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sfi():
    return load_sfi()


def lengths(batch, ranges, context, seed):
    """Query and key lengths of `batch` sequences, each of a random one of the ranges; every third
    has up to `context` keys before its queries."""
    r = random.Random(seed)
    nq = [r.randint(*r.choice(ranges)) for _ in range(batch)]
    return nq, [n + (r.randint(1, context) if context and i % 3 == 0 else 0) for i, n in enumerate(nq)]


MIXED = [(1, 127), (129, 255), (257, 700)]


@pytest.mark.parametrize("hq,hkv,d,batch,ranges,context", [
    (8, 8, 64, 48, [(2, 200)], 0),  # one tile a (sequence, head), of one or two halves and blocks
    (8, 8, 64, 60, MIXED, 0),
    (8, 8, 128, 60, MIXED, 300),
    (24, 8, 64, 60, MIXED, 300),
    (24, 8, 128, 64, MIXED, 0),
    (32, 8, 64, 64, MIXED, 0),
    (32, 8, 128, 60, MIXED, 300),
    (16, 16, 64, 200, [(1, 3), (129, 140), (255, 257)], 0),  # hardly any time between the tiles
    (16, 16, 128, 200, [(1, 3), (129, 140), (255, 257)], 130),
])
def test_tile_after_tile(sfi, hq, hkv, d, batch, ranges, context):
    nq, nk = lengths(batch, ranges, context, 5 * hq + d)
    cu_q, cu_k = offsets(nq), offsets(nk)
    span = 2 * (128 // (hq // hkv))
    assert hkv * sum(-(-n // span) for n in nq) >= 2 * torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = normal((cu_q[-1], hq, d), BF16, 1), normal((cu_k[-1], hkv, d), BF16, 2), normal((cu_k[-1], hkv, d), BF16, 3)
    lay = sfi.PackedLayout(hq, hkv, d, BF16, ints(cu_q), ints(cu_k), cu_q[-1], cu_k[-1])
    ws = sfi.prefill_workspace(lay)
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    sfi.sfi_prefill_attn(lay, q, k, v, out, lse, ws)
    assert sfi.sfi_read_status(ws) == 0
    rows = set(range(0, cu_q[-1], 83)) | {x for y in cu_q[1::4] for x in (y - 1, y) if x < cu_q[-1]}
    ref, rl, scale, size = P.prefill(f64(q), f64(k), f64(v), cu_q, cu_k, rows)
    at = sorted(rows)
    close(f64(out)[at], ref[at], bf16_tolerance(ref, scale, size, d)[at], "out")
    close_lse(f64(lse)[at], rl[at], size[at], d)
    for _ in range(10):
        again, lse2 = torch.full_like(q, 7.0), torch.full_like(lse, 7.0)
        sfi.sfi_prefill_attn(lay, q, k, v, again, lse2, ws)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert sfi.sfi_read_status(ws) == 0
