"""Shared helpers of the prompt-attention and paged-cache tests."""
import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu", torch.float64).numpy()


def offsets(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def ints(v, device="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=device)


def normal(shape, dtype, seed, device="cuda"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float32).to(dtype).to(device)


def score_error(size, d):
    """Bound on a score's error in natural units: fp32 accumulation of d exact products, in any
    order, off by at most one truncation (2^-23) of the sum of magnitudes a step, and the two
    roundings of scale and exponent argument."""
    return (d + 4) * 2.0 ** -23 * size


def bf16_tolerance(ref, scale, size, d):
    """Elementwise bound for attention whose probabilities and whose output are rounded to bf16
    (half a step, eps / 2, each): sum_j |dp_j| |v_j| + |d out|.  A score off by x moves p by a
    factor within e^(2x) (numerator and sum); exp2 and the fp32 sums add 2^-16 between them
    (2^-22 an exp2; sums of at most 2^16 terms that are mostly far from the worst order)."""
    half = torch.finfo(torch.bfloat16).eps / 2
    move = np.expm1(2 * score_error(size, d))[..., None] + 2.0 ** -16
    rel = half + move + half * move
    return rel * scale + half * (np.abs(ref) + rel * scale) + 2.0 ** -133


def close(got, ref, tol, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], np.broadcast_to(tol, ref.shape)[bad][:4])


def close_lse(got, ref, size, d, what="lse"):
    """-inf exactly where the reference has it; else the score bound, 2^-16 for the sum, 4 ulps."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), what
    fin = np.isfinite(ref)
    tol = score_error(size, d)[fin] + 2.0 ** -16 + 2.0 ** -21 * np.abs(ref[fin])
    close(got[fin], ref[fin], tol, what)


def f32_tolerance(ref, scale, size, d, n, split):
    """Elementwise bound for attention with an fp32 output over n positions.  Scores as above; exp2
    off by 2^-22 twice (numerator and sum); sums in any order, off by one truncation of the sum
    of magnitudes a step, at most n / 8 steps in a warp and 64 across warps and pieces (numerator
    and sum); `split`: p as the sum of two bf16 terms, each off by eps / 2 of what is left."""
    move = np.expm1(2 * score_error(size, d))[..., None] + 2.0 ** -21
    move = move + 2 * (n / 8 + 64) * 2.0 ** -23
    if split:
        move = move + (torch.finfo(torch.bfloat16).eps / 2) ** 2
    return move * (scale + np.abs(ref)) + 2.0 ** -126


def pool_of(lens, page, extra, seed):
    """A fragmented pool for these lengths: (n_pages, page table rows padded with -1)."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    ids = np.random.RandomState(seed).permutation(n_pages)
    width = max(need) + 1
    table, at = np.full((len(lens), width), -1, np.int32), 0
    for b, x in enumerate(need):
        table[b, :x] = ids[at:at + x]
        at += x
    return n_pages, table
