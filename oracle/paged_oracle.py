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


def prefill(q, k, v, cu_q, cu_k, rows=None):
    """Causal attention over packed prompts: q [T, H_q, d], k, v [T_k, H_kv, d].
    Returns out, lse, and the two error scales of `attend`; rows outside every
    sequence, and those that are not in `rows` if it is given, are NaN."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, scale = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, size = np.full((T, Hq), np.nan), np.full((T, Hq), np.nan)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            t = cu_q[b] + i
            if rows is not None and t not in rows:
                continue
            for h in range(Hq):
                K = k[cu_k[b]:cu_k[b + 1], h // G]
                V = v[cu_k[b]:cu_k[b + 1], h // G]
                out[t, h], lse[t, h], scale[t, h], size[t, h] = attend(q[t, h], K, V, i + nk - nq + 1)
    return out, lse, scale, size


def paged(q, k, v, table, lens):
    """One token's attention over a paged cache: q [B, H_q, d], k, v pools
    [n_pages, H_kv, P, d].  Returns out, lse and the error scales of `attend`."""
    B, Hq, d = q.shape
    Hkv, P = k.shape[1:3]
    out, scale = np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    lse, size = np.zeros((B, Hq)), np.zeros((B, Hq))
    for b in range(B):
        n = int(lens[b])
        ids = [int(x) for x in table[b][:-(-n // P)]]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            K = np.concatenate([k[x, g] for x in ids])[:n] if n else np.zeros((0, d))
            V = np.concatenate([v[x, g] for x in ids])[:n] if n else np.zeros((0, d))
            out[b, h], lse[b, h], scale[b, h], size[b, h] = attend(q[b, h], K, V, n)
    return out, lse, scale, size


class Pages:
    """The bookkeeping of a paged cache, one sequence and page at a time: page
    table, lengths, reference counts, and pools [layers, n_pages, H_kv, P, d].
    Every call returns the names of what went wrong ("pages", "index", "len")."""

    def __init__(self, table, lens, ref, k, v):
        self.table, self.len, self.ref = np.array(table), np.array(lens), np.array(ref)
        self.k, self.v = np.array(k), np.array(v)
        self.P = self.k.shape[3]

    def held(self, b):
        return -(-int(self.len[b]) // self.P)

    def lowest_free(self):
        free = np.nonzero(self.ref == 0)[0]
        return int(free[0]) if len(free) else None

    def extend(self, n_new):
        bad = set()
        left = int((self.ref == 0).sum())
        for b, more in enumerate(n_new):
            if more < 0:
                bad.add("len")
                continue
            want = -(-(int(self.len[b]) + more) // self.P) - self.held(b)
            if want > left or int(self.len[b]) + more > self.table.shape[1] * self.P:
                bad.add("pages")
                continue
            left -= want
            for i in range(want):
                x = self.lowest_free()
                self.table[b, self.held(b) + i] = x
                self.ref[x] = 1
            self.len[b] += more
        return bad

    def fork(self, src, dst):
        bad = set()
        for s, t in zip(src, dst):
            n = int(self.len[s])
            if self.len[t] != 0:
                bad.add("index")
                continue
            full, part = n // self.P, n % self.P
            x = self.lowest_free() if part else None
            if part and x is None:
                bad.add("pages")
                continue
            self.table[t, :full] = self.table[s, :full]
            for i in range(full):
                self.ref[self.table[s, i]] += 1
            if part:
                self.table[t, full] = x
                self.ref[x] = 1
                for pool in (self.k, self.v):
                    pool[:, x, :, :part] = pool[:, self.table[s, full], :, :part]
            self.len[t] = n
        return bad

    def free(self, seqs):
        bad = set()
        for b in seqs:
            for i in range(self.held(b)):
                x = self.table[b, i]
                if self.ref[x] <= 0:
                    bad.add("index")
                else:
                    self.ref[x] -= 1
                self.table[b, i] = -1
            self.len[b] = 0
        return bad

    def compact(self):
        n = len(self.ref)
        live = int((self.ref > 0).sum())
        to = np.where(self.ref > 0, np.arange(n), -1)
        holes = [x for x in range(live) if self.ref[x] == 0]
        moved = [x for x in range(live, n) if self.ref[x] > 0]
        for a, b in zip(moved, holes):
            to[a] = b
            self.ref[b], self.ref[a] = self.ref[a], 0
            for pool in (self.k, self.v):
                pool[:, b] = pool[:, a]
        for b in range(len(self.len)):
            for i in range(self.held(b)):
                self.table[b, i] = to[self.table[b, i]]
        return to

    def append(self, layer, k_new, v_new, cu):
        for b in range(len(self.len)):
            m = cu[b + 1] - cu[b]
            for i in range(m):
                pos = int(self.len[b]) - m + i
                x = self.table[b, pos // self.P]
                self.k[layer, x, :, pos % self.P] = k_new[cu[b] + i]
                self.v[layer, x, :, pos % self.P] = v_new[cu[b] + i]
