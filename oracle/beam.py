"""Oracle: one step of beam search over beams and vocabulary, and the beams' paged cache; fp64 and plain loops.

Beam j of a request offers every token with score + log_softmax(row / tau), or, once finished, itself only.
Continuations are ranked by score / ((5 + length) / 6)^alpha (the length penalty of Wu et al. 2016, "Google's
Neural Machine Translation System", section 7, without its coverage term); ties go to the lower beam, then the
lower token.
"""
import numpy as np


def offers(row, score, length, finished, tau, alpha, eos):
    """(rank, token, score, length, finished) of everything that one beam offers."""
    if not score > -np.inf:
        return []
    if finished:
        token = eos if 0 <= eos < len(row) else 0
        return [(score / ((5 + length) / 6) ** alpha, token, score, length, 1)]
    x = np.asarray(row, dtype=np.float64) / tau
    if np.isnan(x).any() or np.isposinf(x).any() or not np.isfinite(x).any():
        return []
    m = x.max()
    logp = (x - m) - np.log(np.exp(x - m).sum())       # (in this order a row of lowest values keeps its logarithm)
    pen = ((5 + length + 1) / 6) ** alpha
    return [((score + p) / pen, t, score + p, length + 1, int(t == eos)) for t, p in enumerate(logp) if p > -np.inf]


def select(logits, scores, lengths, finished, tau, alpha, eos):
    """logits [B, W, V]; the others [B, W].  Returns parent, token, score, length, finished [B, W] and each
    request's list of all ranks, largest first."""
    B, W, _ = logits.shape
    parent, token, length, done = (np.zeros((B, W), dtype=int) for _ in range(4))
    score, ranks = np.zeros((B, W)), []
    for b in range(B):
        every = []
        for j in range(W):
            every += [(o[0], j) + o[1:] for o in offers(logits[b, j], float(scores[b, j]), int(lengths[b, j]), bool(finished[b, j]), tau, alpha, eos)]
        every.sort(key=lambda o: (-o[0], o[1], o[2]))
        ranks.append([o[0] for o in every])
        for j in range(W):
            if j < len(every):
                _, parent[b, j], token[b, j], score[b, j], length[b, j], done[b, j] = every[j]
            else:
                parent[b, j], token[b, j], score[b, j], length[b, j], done[b, j] = j, 0, -np.inf, lengths[b, j], 0
    return parent, token, score, length, done, ranks


def reorder(table, kv_len, parent, bs, num_blocks):
    """table [B * W, n].  Returns the new table, the copies as (request, from page, to page, rows) and the
    status of each request: 0, 1 (a parent outside [0, W)), 2 (length), 32 (a writing page)."""
    table = np.array(table)
    new, copies, status = table.copy(), [], []
    W = len(parent[0])
    for b, L in enumerate(kv_len):
        rows = range(b * W, b * W + W)
        page, rem = L // bs, L % bs
        if any(not 0 <= p < W for p in parent[b]):
            status.append(1)
            continue
        if L < 0 or page >= table.shape[1]:
            status.append(2)
            continue
        writing = [int(table[r, page]) for r in rows]
        if any(not 0 <= p < num_blocks for p in writing) or len(set(writing)) < W:
            status.append(32)
            continue
        status.append(0)
        free = [writing[j] for j in range(W) if j not in list(parent[b])]
        met = set()
        for j, p in enumerate(parent[b]):
            new[b * W + j, :page] = table[b * W + p, :page]
            if p in met:
                to = free.pop(0)
                if rem:
                    copies.append((b, writing[p], to, rem))
            else:
                to = writing[p]
                met.add(p)
            new[b * W + j, page] = to
    return new, copies, status
