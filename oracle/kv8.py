"""The 8-bit K/V cache in plain numpy, fp64: e4m3 codes with one scale per (block, KV head).

Codes are handled as the values they stand for (float64 arrays of e4m3 values); a cached value is
code * scale.  Written from the definitions in include/spec_verify.h, element by element where a
loop is clearer than indexing.
"""
import numpy as np

E4M3_MAX = 448.0
S_MIN, S_MAX = 2.0 ** -100, 2.0 ** 119


def e4m3_values():
    """The value of each of the 256 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits; the
    all-ones pattern is NaN, there are no infinities)."""
    out = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 128 else 1.0
        e, m = (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


def round_e4m3(x):
    """Nearest e4m3 value, ties to even, saturating at 448 (infinities too); NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    y = np.clip(x, -E4M3_MAX, E4M3_MAX)
    _, e = np.frexp(np.where(np.isnan(y), 0.0, y))      # |y| = f 2^e, f in [1/2, 1)
    step = 2.0 ** (np.maximum(e - 1, -6) - 3.0)
    return np.where(np.isnan(x), np.nan, np.rint(y / step) * step)


def need_scale(a):
    """Smallest power of two s with a <= 448 s, in [2^-100, 2^119]."""
    s = S_MIN
    while a > E4M3_MAX * s and s < S_MAX:
        s *= 2
    return s


def _f32(x):
    return float(np.float32(x))


def append(codes, scale, x, table, start, row_offset, bs, status=None):
    """One cache (K or V): codes [num_blocks, H, bs, d] and scale [num_blocks, H] are updated in
    place with the rows x [N, H, d]; returns the status bits added per request."""
    num_blocks, H = scale.shape
    N = x.shape[0]
    added = [0] * len(start)
    top = int(row_offset[0])                            # the largest offset so far
    for r in range(len(start)):
        o, o1, p0 = int(row_offset[r]), int(row_offset[r + 1]), int(start[r])
        bad = o < 0 or o1 < o or o1 > N or o < top or p0 < 0 or p0 + o1 - o > 2 ** 31 - 1
        top = max(top, o, o1)
        if status is not None and int(status[r]) & ~32:
            continue
        if bad:
            added[r] |= 2
            continue
        t = 0
        while t < o1 - o:
            slot = p0 + t
            row = slot % bs
            n = min(bs - row, o1 - o - t)
            lb = slot // bs
            b = int(table[r][lb]) if lb < len(table[r]) else -1
            if b < 0 or b >= num_blocks:
                added[r] |= 32
                t += n
                continue
            for h in range(H):
                new = x[o + t:o + t + n, h].astype(np.float64)
                fin = np.abs(new[np.isfinite(new)])
                s = need_scale(float(fin.max()) if fin.size else 0.0)
                if row:
                    old = float(scale[b, h])
                    s = max(old, s)
                    if s > old:
                        ratio = _f32(old / s)
                        codes[b, h, :row] = round_e4m3((codes[b, h, :row] * ratio).astype(np.float32))
                codes[b, h, row:row + n] = round_e4m3((new / s).astype(np.float32))
                scale[b, h] = s
            t += n
    return added


def compact(codes, scale, table, prefix, path, n_acc, bs):
    """One layer's cache (K or V), in place; requests with n_acc < 0 are left alone."""
    was, at = codes.copy(), scale.copy()
    H = scale.shape[1]
    for r in range(len(prefix)):
        P, na = int(prefix[r]), int(n_acc[r])
        if na < 0:
            continue
        moves = [(P + int(path[r][d]), P + d) for d in range(na + 1)]
        for lb in sorted({b // bs for _, b in moves}):
            mine = [(a, b) for a, b in moves if b // bs == lb]
            if all(a == b for a, b in mine):
                continue
            to, kept = int(table[r][lb]), max(0, min(bs, P - lb * bs))
            for h in range(H):
                s = max([at[int(table[r][a // bs]), h] for a, _ in mine]
                        + ([at[to, h]] if kept else []))
                def put(row, src_block, src_row):
                    ratio = _f32(at[src_block, h] / s)
                    codes[to, h, row] = round_e4m3((was[src_block, h, src_row] * ratio).astype(np.float32))
                for row in range(kept):
                    put(row, to, row)
                for a, b in mine:
                    put(b % bs, int(table[r][a // bs]), a % bs)
                scale[to, h] = s


def tree_attention(q, k, ks, v, vs, table, prefix, node_offset, visible, bs, scale=None):
    """q [N, H_q, d]; k, v [num_blocks, H, bs, d] code values, ks, vs [num_blocks, H]; visible[n] =
    bool array over the tree slots of n's request.  Returns (o, lse, mass, err): mass is the mean
    absolute value sum p|v| / sum p and err the inputs of the tests' tolerances: per row the largest
    over visible keys of scale * (max|q| * sum|k|, sum|q k|), and sum|v| over sum p / max p."""
    N, Hq, d = q.shape
    H = ks.shape[1]
    G = Hq // H
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o = np.zeros((N, Hq, d))
    lse = np.full((N, Hq), -np.inf)
    mass = np.zeros((N, Hq, d))
    err = np.zeros((N, Hq, 2))
    tail = np.zeros((N, Hq, d))
    for r in range(len(prefix)):
        P, o0, o1 = int(prefix[r]), int(node_offset[r]), int(node_offset[r + 1])
        S = P + o1 - o0
        if o1 <= o0:
            continue
        ids = np.asarray([int(b) for b in table[r][:-(-S // bs)]], dtype=np.int64)
        for h in range(H):
            kk = (k[ids, h] * ks[ids, h][:, None, None]).reshape(-1, d)[:S]
            vv = (v[ids, h] * vs[ids, h][:, None, None]).reshape(-1, d)[:S]
            for n in range(o0, o1):
                keep = np.concatenate([np.ones(P, dtype=bool), np.asarray(visible[n][:o1 - o0], dtype=bool)])
                if not keep.any():
                    continue
                kn, vn = kk[keep], vv[keep]
                for g in range(h * G, (h + 1) * G):
                    x = kn @ q[n, g] * scale
                    m = x.max()
                    p = np.exp(x - m)
                    o[n, g] = p @ vn / p.sum()
                    mass[n, g] = p @ np.abs(vn) / p.sum()
                    lse[n, g] = m + np.log(p.sum())
                    err[n, g, 0] = scale * np.abs(q[n, g]).max() * np.abs(kn).sum(axis=1).max()
                    err[n, g, 1] = scale * (np.abs(kn) @ np.abs(q[n, g])).max()
                    tail[n, g] = np.abs(vn).sum(axis=0) / p.sum()
    return o, lse, mass, err, tail
