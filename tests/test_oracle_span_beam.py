"""Pins of the oracles of windowed and shared-prefix attention and of beam search: library attention with
explicit masks, library log-softmax, exhaustive search, and a cache rebuilt token by token."""
import itertools

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import beam, span


def _case(prefix, sizes, rng, H=2, G=2, d=8, bs=4, chain=True):
    need = [-(-(p + t) // bs) for p, t in zip(prefix, sizes)]
    ids = rng.permutation(sum(need) + 2)
    table, at = np.full((len(need), max(need)), -1), 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    k, v = rng.normal(size=(2, len(ids), H, bs, d))
    off = np.concatenate([[0], np.cumsum(sizes)])
    bits, parents = [], []
    for T in sizes:
        mine = []
        for i in range(T):
            p = i - 1 if chain else (-1 if i == 0 else int(rng.integers(0, i)))
            mine.append((mine[p] if p >= 0 else 0) | (1 << i))
            parents.append(p)
        bits += mine
    return k, v, table, off, bits, parents, rng.normal(size=(int(off[-1]), H * G, d))


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (5, 1), (100, 0), (2, 100)])
def test_window_of_a_chain_is_banded_library_attention(window, sinks):
    rng = np.random.default_rng(window * 7 + sinks)
    k, v, table, off, bits, _, q = _case([9, 0], [5, 6], rng)
    o, lse, _, _ = span.attention(q, k, v, table, [9, 0], off, bits, 4, window=window, sinks=sinks)
    for r, P in enumerate([9, 0]):
        T = [5, 6][r]
        slots = np.arange(P + T)
        K = torch.from_numpy(k[table[r][slots // 4], :, slots % 4]).permute(1, 0, 2).repeat_interleave(2, 0)
        V = torch.from_numpy(v[table[r][slots // 4], :, slots % 4]).permute(1, 0, 2).repeat_interleave(2, 0)
        i, j = np.arange(P, P + T)[:, None], slots[None, :]
        seen = torch.from_numpy((j <= i) & ((i - j < window) | (j < sinks)))
        Q = torch.from_numpy(q[off[r]:off[r + 1]]).permute(1, 0, 2)
        want = torch.nn.functional.scaled_dot_product_attention(Q, K, V, attn_mask=seen).permute(1, 0, 2).numpy()
        np.testing.assert_allclose(o[off[r]:off[r + 1]], want, atol=1e-12)
        x = (Q @ K.transpose(1, 2) / np.sqrt(8)).masked_fill(~seen, -np.inf)
        np.testing.assert_allclose(lse[off[r]:off[r + 1]], torch.logsumexp(x, 2).T.numpy(), atol=1e-12)


def test_wide_window_and_own_groups_are_tree_attention():
    rng = np.random.default_rng(1)
    k, v, table, off, bits, parents, q = _case([7, 3, 0], [6, 1, 9], rng, chain=False)
    want = A.tree_attention(q, k, v, table, [7, 3, 0], off, parents, 4)
    for kw in (dict(window=16), dict(window=1, sinks=99), dict(groups=[(0, 1, 7), (1, 2, 0), (2, 3, 0)])):
        o, lse, _, _ = span.attention(q, k, v, table, [7, 3, 0], off, bits, 4, **kw)
        np.testing.assert_allclose(o, want["o"], atol=1e-12)
        np.testing.assert_allclose(lse, want["lse"], atol=1e-12)


def test_window_goes_by_depth_not_by_slot():
    # root, two children, a grandchild of the second: slots 0 .. 3, depths 0 1 1 2
    bits = [1, 3, 5, 13]
    assert span.visible(bits[3], 10, 4, window=1) == [13]
    assert span.visible(bits[3], 10, 4, window=2) == [12, 13]
    assert span.visible(bits[3], 10, 4, window=3) == [10, 12, 13]
    assert span.visible(bits[3], 10, 4, window=4) == [9, 10, 12, 13]
    assert span.visible(bits[3], 10, 4, window=1, sinks=2) == [0, 1, 13]
    assert span.visible(bits[3], 1, 4, window=1, sinks=3) == [0, 1, 3, 4]    # sinks reach into the tree
    # an empty row stands at position P
    assert span.visible(0, 2, 4, window=1) == [] and span.visible(0, 2, 4, window=2) == [1] and span.visible(0, 0, 4) == []


def test_shared_slots_come_from_the_first_request():
    rng = np.random.default_rng(2)
    k, v, table, off, bits, _, q = _case([10, 8, 9], [1, 2, 1], rng)
    same = table.copy()
    for r in (1, 2):       # what the members' own pages hold of the first 6 slots does not count
        for s in range(6):
            k[same[r][s // 4], :, s % 4] = np.nan
    o, lse, _, _ = span.attention(q, k, v, table, [10, 8, 9], off, bits, 4, groups=[(0, 3, 6)])
    for r in (1, 2):
        for s in range(6):
            k[same[r][s // 4], :, s % 4] = k[table[0][s // 4], :, s % 4]
            v[same[r][s // 4], :, s % 4] = v[table[0][s // 4], :, s % 4]
    want, wl, _, _ = span.attention(q, k, v, table, [10, 8, 9], off, bits, 4)
    np.testing.assert_allclose(o, want, atol=1e-12)
    np.testing.assert_allclose(lse, wl, atol=1e-12)


@pytest.mark.parametrize("alpha,tau", [(0.0, 1.0), (0.6, 0.7), (1.0, 1.3)])
def test_select_against_exhaustive_search(alpha, tau):
    rng = np.random.default_rng(3)
    B, W, V, eos = 4, 3, 6, 2
    x, s = rng.normal(size=(B, W, V)) * 2, -rng.random((B, W)) * 3
    length, done = rng.integers(1, 9, (B, W)), rng.random((B, W)) < 0.4
    parent, token, score, n, fin, _ = beam.select(x, s, length, done, tau, alpha, eos)
    logp = torch.log_softmax(torch.from_numpy(x) / tau, dim=2).numpy()
    for b in range(B):
        every = []
        for j, t in itertools.product(range(W), range(V)):
            if done[b, j]:
                if t != eos:
                    continue
                every.append((s[b, j] / ((5 + length[b, j]) / 6) ** alpha, j, t, s[b, j], length[b, j], 1))
            else:
                v = s[b, j] + logp[b, j, t]
                every.append((v / ((6 + length[b, j]) / 6) ** alpha, j, t, v, length[b, j] + 1, int(t == eos)))
        best = sorted(every, key=lambda e: -e[0])[:W]
        for k, (_, j, t, v, ln, f) in enumerate(best):
            assert (parent[b, k], token[b, k], n[b, k], fin[b, k]) == (j, t, ln, f)
            assert abs(score[b, k] - v) < 1e-12


def test_select_of_width_one_is_greedy_and_ties_go_low():
    x = np.zeros((1, 1, 5))
    assert beam.select(x, np.zeros((1, 1)), np.ones((1, 1), int), np.zeros((1, 1)), 1.0, 0.0, -1)[1][0, 0] == 0
    parent, token, *_ = beam.select(np.zeros((1, 3, 4)), np.zeros((1, 3)), np.ones((1, 3), int), np.zeros((1, 3)), 1.0, 0.0, -1)
    assert parent.tolist() == [[0, 0, 0]] and token.tolist() == [[0, 1, 2]]


def test_select_with_unused_beams_and_broken_rows():
    x = np.zeros((1, 3, 2))
    x[0, 1, 0] = np.nan
    s = np.array([[-np.inf, 0.0, -1.0]])
    parent, token, score, n, fin, _ = beam.select(x, s, np.full((1, 3), 4), np.zeros((1, 3)), 1.0, 0.0, -1)
    assert parent.tolist() == [[2, 2, 2]] and token.tolist() == [[0, 1, 0]]
    assert np.isneginf(score[0, 2]) and n.tolist() == [[5, 5, 4]]


def test_reorder_keeps_every_beams_tokens():
    """A cache that holds each slot's history: after any run of reorderings beam j's pages read as its own
    sequence of tokens, and the writing pages stay distinct."""
    rng = np.random.default_rng(4)
    B, W, bs, n = 2, 4, 3, 8
    nb = B * W * n
    table = rng.permutation(nb).reshape(B * W, n)
    cache = np.full((nb, bs), -1)
    lens = [2, 5]
    want = [[list(range(100 * b, 100 * b + L)) for _ in range(W)] for b, L in enumerate(lens)]
    for b in range(B):
        for j in range(W):
            for s, t in enumerate(want[b][j]):
                cache[table[b * W + j, s // bs], s % bs] = t
    for step in range(12):
        for b in range(B):
            for j in range(W):
                tok = 1000 + 100 * step + 10 * b + j
                cache[table[b * W + j, lens[b] // bs], lens[b] % bs] = tok
                want[b][j].append(tok)
            lens[b] += 1
        parent = rng.integers(0, W, (B, W))
        table, copies, status = beam.reorder(table, lens, parent, bs, nb)
        assert status == [0, 0]
        for _, fr, to, rem in copies:
            cache[to, :rem] = cache[fr, :rem]
        for b in range(B):
            want[b] = [list(want[b][p]) for p in parent[b]]
            for j in range(W):
                assert [cache[table[b * W + j, s // bs], s % bs] for s in range(lens[b])] == want[b][j]
            page = lens[b] // bs
            assert len({table[b * W + j, page] for j in range(W)}) == W


def test_reorder_statuses():
    t = np.array([[0, 1], [2, 3], [4, 5], [4, 5], [6, 99], [7, 8]])
    new, copies, status = beam.reorder(t, [1, 2, 3], [[0, 2], [0, 1], [0, 0]], 2, 50)
    assert status == [1, 32, 32] and (new == t).all() and copies == []
    assert beam.reorder(t, [4, -1, 0], [[0, 1], [0, 1], [1, 1]], 2, 50)[2] == [2, 2, 0]
