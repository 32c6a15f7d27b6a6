"""fp64 restatement of the prompt attention and of the paged KV cache: plain
loops over sequences, heads and pages, written from the definitions; shares no
code with the GPU path."""
import numpy as np


def attend(q, K, V, limit):
    """One query row [d] over the first `limit` rows of K, V [n, d]:
    (out [d], ln sum exp, sum_j p_j |v_j| [d], max_j sum |q||k_j| / sqrt(d))."""
    d = q.shape[0]
    if limit <= 0:
        return np.zeros(d), -np.inf, np.zeros(d), 0.0
    s = K[:limit] @ q / np.sqrt(d)
    m = s.max()
    e = np.exp(s - m)
    p = e / e.sum()
    size = float(np.max(np.abs(K[:limit]) @ np.abs(q))) / np.sqrt(d)
    return p @ V[:limit], m + np.log(e.sum()), p @ np.abs(V[:limit]), size


def prefill(q, k, v, cu_q, cu_k):
    """Causal attention over packed prompts: q [T, H_q, d], k, v [T_k, H_kv, d].
    Returns out, lse, and the two error scales of `attend`; rows outside every
    sequence are NaN."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, scale = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, size = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            t = cu_q[b] + i
            for h in range(Hq):
                K = k[cu_k[b]:cu_k[b + 1], h // G]
                V = v[cu_k[b]:cu_k[b + 1], h // G]
                out[t, h], lse[t, h], scale[t, h], size[t, h] = attend(q[t, h], K, V, i + nk - nq + 1)
    return out, lse, scale, size
