"""64-bit restatement of the norm and rotation of heads and of the 8-bit rows of a
paged cache, written from the definitions; shares no code with the GPU path."""
import numpy as np

TWO_PI = np.longdouble("6.283185307179586476925286766559005768394")


def norm_rope(x, w, pos, inv_freq, interleaved, eps):
    """x [rows, heads, d]; w [d] or None; eps None: no norm.  Returns the rotated heads and, for
    each element, the sum of magnitudes of the terms that make it."""
    rows, heads, d = x.shape
    n = x.astype(np.float64)
    if eps is not None:
        n = n / np.sqrt((n * n).sum(-1, keepdims=True) / d + eps)
        if w is not None:
            n = n * w
    out, size = n.copy(), np.abs(n)
    r = 2 * len(inv_freq)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        for t in range(rows):
            angle = np.fmod(np.longdouble(int(pos[t])) * np.longdouble(f), TWO_PI)
            c, s = np.cos(angle), np.sin(angle)
            out[t, :, a] = (n[t, :, a] * c - n[t, :, b] * s).astype(np.float64)
            out[t, :, b] = (n[t, :, a] * s + n[t, :, b] * c).astype(np.float64)
            size[t, :, a] = size[t, :, b] = np.abs(n[t, :, a]) + np.abs(n[t, :, b])
    return out, size


def quantise(x, fmt):
    """Rows [..., d] of fp32 numbers as 8-bit codes (the numbers that they are, float64) and fp32
    scales.  A quotient of two fp32 numbers that is not a tie of 8 bits is too far from one for
    64 bits to take it for one."""
    x = np.asarray(x, np.float32)
    codes, scales = np.zeros(x.shape), np.zeros(x.shape[:-1], np.float32)
    with np.errstate(all="ignore"):
        for at in np.ndindex(*x.shape[:-1]):
            row = x[at].astype(np.float64)
            if not np.isfinite(row).all():
                scales[at] = np.nan
                continue
            top = np.abs(row).max()
            if fmt == "i8":
                s = np.float32(np.float32(top) / np.float32(127))
            else:
                s = np.float32(0)
                for k in range(max(-149, int(np.floor(np.log2(top))) - 10), 121) if top > 0 else ():
                    if top <= 448 * 2.0 ** k:
                        # (below 2^-149 there is no scale: the smallest power of two for the row would be one)
                        if k > -149 or top > 448 * 2.0 ** -150:
                            s = np.float32(2.0 ** k)
                        break
            scales[at] = s
            if s == 0:
                continue
            y = row / np.float64(s)
            if fmt == "i8":
                codes[at] = np.clip(np.rint(y), -127, 127)
            else:
                step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
                codes[at] = np.rint(y / step) * step
    return codes, scales
