"""Oracle: tree attention with a sliding window and sinks, and under prefixes that requests share; fp64.

No page gives formulas for either; both are oracle.attention's tree attention with another set of visible
slots, or another place where some slots are kept:
  window  node i at position m = P + depth(i) sees the token at position p iff p < sinks or m - p < window;
          prefix slot s is at position s, a node's k-th ancestor-or-self (in increasing index) at P + k
  shared  the first `length` slots of a group's requests are read through its first request's table row
`bits[n]` is node n's row of the ancestor mask as an integer (bit a: tree node a).
"""
import numpy as np


def members(bits, T):
    return [a for a in range(T) if (bits >> a) & 1]


def visible(bits, P, T, window=None, sinks=0):
    """The logical slots that a node with these mask bits sees."""
    own = members(bits, T)
    if window is None:
        return list(range(P)) + [P + a for a in own]
    m = P + max(len(own) - 1, 0)
    near = lambda p: p < sinks or m - p < window  # noqa: E731
    return [s for s in range(P) if near(s)] + [P + a for k, a in enumerate(own) if near(P + k)]


def attention(q, k_cache, v_cache, table, prefix, offset, bits, bs, scale=None, window=None, sinks=0, groups=None):
    """q [N, H_q, d], caches [num_blocks, H_kv, bs, d]; groups: list of (first request, end, length).

    Returns o [N, H_q, d] and lse [N, H_q] (0 and -inf for a row that sees nothing), the sums of weight
    times |v| as o, and the largest sum of |q_c k_c| times the scale of a row's keys as lse.
    """
    N, H_q, d = q.shape
    G = H_q // k_cache.shape[1]
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, mass = np.zeros((N, H_q, d)), np.zeros((N, H_q, d))
    lse, size = np.full((N, H_q), -np.inf), np.zeros((N, H_q))
    for r, P in enumerate(prefix):
        lo, T = int(offset[r]), int(offset[r + 1] - offset[r])
        first, length = r, 0
        for a, b, n in groups or []:
            if a <= r < b:
                first, length = a, n
        for i in range(T):
            slots = np.array(visible(bits[lo + i], P, T, window, sinks), dtype=int)
            if len(slots) == 0:
                continue
            page = np.where(slots < length, table[first][np.minimum(slots // bs, table.shape[1] - 1)], table[r][slots // bs])
            for h in range(H_q):
                K, V = k_cache[page, h // G, slots % bs], v_cache[page, h // G, slots % bs]
                x = K @ q[lo + i, h] * scale
                w = np.exp(x - x.max())
                o[lo + i, h] = w @ V / w.sum()
                mass[lo + i, h] = w @ np.abs(V) / w.sum()
                lse[lo + i, h] = x.max() + np.log(w.sum())
                size[lo + i, h] = (np.abs(K) @ np.abs(q[lo + i, h])).max() * abs(scale)
    return o, lse, mass, size
