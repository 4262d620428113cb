"""GPU parity of beam selection and of the beams' cache with the fp64 oracle, and a whole search."""
import numpy as np
import pytest
import torch

import kv8_util as U
from oracle import beam
from speculative_decoding_draft_tree_gb300 import binding as B
from speculative_decoding_draft_tree_gb300.api import BeamSearch

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------------------------------ select
class Select:
    def __init__(self, x, scores, lengths, finished, V, tau=1.0, alpha=0.0, eos=-1, dtype=F32, pad=8):
        self.B, self.W = scores.shape
        ld = -(-V // 8) * 8 + pad
        self.rows = torch.full((self.B * self.W, ld), float("nan"), dtype=dtype, device="cuda")     # padding is not read
        self.rows[:, :V] = torch.from_numpy(np.asarray(x, dtype=np.float64)).reshape(self.B * self.W, V).cuda().to(dtype)
        self.scores = torch.from_numpy(np.asarray(scores)).float().cuda()
        self.lengths, self.finished = U.ints(np.asarray(lengths).tolist()), U.ints(np.asarray(finished).astype(int).tolist())
        self.V, self.tau, self.alpha, self.eos = V, tau, alpha, eos
        shape = dict(size=(self.B, self.W), device="cuda")
        self.out = [torch.full(**shape, fill_value=-9, dtype=t) for t in (torch.int32, torch.int32, F32, torch.int32, torch.int32)]

    def params(self, out=None):
        o = out or self.out
        return B.beam_select_params(self.rows, self.V, self.tau, self.scores, self.lengths, self.finished, self.eos, self.alpha, *o)

    def run(self, out=None, stream=None):
        p = self.params(out)
        ws = torch.full((max(256, B.spec_beam_select_workspace_size(p)),), 0xA5, dtype=torch.uint8, device="cuda")
        B.spec_beam_select(p, ws, stream)
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (out or self.out)]

    def check(self):
        """Per thread a sum of exponentials in fp32, in groups of 32 or 16: at most V / 256 + 64 roundings of 2^-24
        and 2^-22 for an exponential, whatever the split; log p and the score are exact beyond that but for
        one rounding of log2(e) / tau (2^-24 of log p) and of the score (2^-24).  Ranks divide by a penalty of
        at least (5 / 6)^alpha.  Choices are the oracle's wherever its ranks lie further apart than that."""
        x = self.rows[:, :self.V].double().cpu().numpy().reshape(self.B, self.W, self.V)
        before = [t.cpu().numpy() for t in (self.scores, self.lengths, self.finished)]
        want = beam.select(x, *before, self.tau, self.alpha, self.eos)
        got = self.run()
        sums = (self.V / 256 + 64) * 2.0 ** -24 + 2.0 ** -21
        for b in range(self.B):
            ranks = np.array(want[5][b][:self.W + 1] + [-np.inf])
            near = sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(ranks), ranks, 0)).max() + 2.0 ** -22 * 40
            near *= 1.2 ** self.alpha
            clear = np.append(ranks[:-1] - ranks[1:] > 2 * near, True)
            for j in range(self.W):
                settled = (j == 0 or clear[j - 1]) and clear[j] if j + 1 < len(ranks) else True
                tied = j + 1 < len(ranks) and ranks[j] == ranks[j + 1]
                if settled or (tied and np.unique(x[b]).size < 3):
                    for k in (0, 1, 3, 4):
                        assert got[k][b, j] == want[k][b, j], (b, j, k, ranks)
                if np.isfinite(want[2][b, j]):
                    assert abs(got[2][b, j] - want[2][b, j]) <= 3 * near + 2.0 ** -23 * abs(want[2][b, j])
                else:
                    assert np.isneginf(got[2][b, j])
        return got, want


def _inputs(B_, W, V, seed, done=0.2):
    rng = np.random.default_rng(seed)
    return rng.normal(size=(B_, W, V)) * 3, -np.cumsum(rng.random((B_, W)), axis=1) * 2, rng.integers(1, 50, (B_, W)), rng.random((B_, W)) < done


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B_,W,V", [(1, 1, 1), (1, 4, 1), (3, 2, 2), (2, 16, 3), (5, 3, 7), (1, 16, 50), (70, 5, 257), (2, 8, 4097), (1, 4, 32000), (3, 7, 50257), (40, 16, 2000)])
def test_select_shapes(B_, W, V, dtype):
    Select(*_inputs(B_, W, V, V + W), V, eos=min(2, V - 1), dtype=dtype).check()


@pytest.mark.parametrize("tau,alpha", [(0.3, 0.0), (2.5, 0.6), (1.0, 1.0), (0.8, 2.0)])
def test_select_temperature_and_length_penalty(tau, alpha):
    Select(*_inputs(6, 5, 3001, 9), 3001, tau=tau, alpha=alpha, eos=17).check()


def test_select_large_vocabulary():
    Select(*_inputs(2, 4, 152064, 1), 152064, eos=3, dtype=BF16).check()
    Select(*_inputs(1, 2, 152063, 2), 152063, eos=3).check()


@pytest.mark.parametrize("V", [5, 700, 40000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_select_ties_go_to_the_lower_beam_and_token(V, dtype):
    """All logits alike: more candidates reach the bound than the list holds."""
    got, _ = Select(np.full((2, 6, V), -1.5), np.zeros((2, 6)), np.full((2, 6), 3), np.zeros((2, 6)), V, dtype=dtype).check()
    assert got[0].tolist() == [[j // V for j in range(6)]] * 2 and got[1].tolist() == [[j % V for j in range(6)]] * 2
    # one better token behind them
    x = np.full((1, 3, V), 0.25)
    x[0, :, V - 1] = 4
    got, _ = Select(x, np.array([[0.0, -1, -30]]), np.full((1, 3), 3), np.zeros((1, 3)), V, dtype=dtype).check()
    assert got[1][0, 0] == V - 1 and got[0][0].tolist()[:2] == [0, 1]


def test_select_zeros_of_both_signs_are_a_tie():
    """Finished beams of score -0 and 0, and logits of both, go by beam and token."""
    x = np.zeros((1, 4, 8))
    x[0, 3] = [-np.inf, -0.0, 0.0, -0.0, -np.inf, -np.inf, -np.inf, -np.inf]
    got = Select(x, np.array([[-0.0, 0.0, -0.0, -1.0]]), [[3, 3, 3, 3]], [[1, 1, 1, 0]], 8, eos=7).run()
    assert got[0].tolist() == [[0, 1, 2, 3]] and got[1].tolist() == [[7, 7, 7, 1]]


def test_select_equal_values_at_the_bound():
    """Two values only: the larger one in fewer places than W, then ties in order."""
    V = 9000
    x = np.zeros((1, 8, V))
    x[0, 0, [8999, 17, 4000]] = 9
    got, _ = Select(x, np.where(np.arange(8) == 0, 0.0, -90.0)[None], np.full((1, 8), 3), np.zeros((1, 8)), V, dtype=BF16).check()
    assert got[1][0].tolist() == [17, 4000, 8999, 0, 1, 2, 3, 4]


def test_select_minus_infinity_nan_and_unused_beams():
    V = 500
    x, s, n, _ = _inputs(7, 4, V, 3, 0)
    x[0, 0] = -np.inf                       # offers nothing
    x[1, 1, 100:] = -np.inf
    x[2, 2, 7] = np.nan                     # out
    x[3, 0, 9] = np.inf                     # out
    x[4, :, 2:] = -np.inf                   # two tokens a beam
    s[5, 1:] = -np.inf                      # the first step: one beam in use
    s[6] = -np.inf                          # nothing at all
    s[2, 3] = np.nan
    for dtype in (F32, BF16):
        got, _ = Select(x, s, n, np.zeros((7, 4)), V, eos=1, dtype=dtype).check()
        assert got[0][6].tolist() == [0, 1, 2, 3] and np.isneginf(got[2][6]).all() and (got[3][6] == n[6]).all()
        assert (got[0][5] == 0).all() and not (got[0][2] >= 2).any() and not (got[0][3] == 0).any()


def test_select_fewer_continuations_than_beams():
    x = np.zeros((1, 5, 2))
    s = np.array([[-1.0, -np.inf, -np.inf, -2.0, -np.inf]])
    got, _ = Select(x, s, np.full((1, 5), 7), np.array([[0, 0, 0, 1, 0]]), 2, eos=1).check()
    assert got[0].tolist() == [[0, 0, 3, 3, 4]] and got[1].tolist() == [[0, 1, 1, 0, 0]]
    assert got[3].tolist() == [[8, 8, 7, 7, 7]] and got[4].tolist() == [[0, 1, 1, 0, 0]]


def test_select_in_place_on_a_stream_and_in_a_graph():
    c = Select(*_inputs(4, 4, 900, 5), 900, eos=2)
    want = c.run()
    s0, l0, f0 = c.scores.clone(), c.lengths.clone(), c.finished.clone()
    out = [c.out[0], c.out[1], c.scores, c.lengths, c.finished]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = c.run(out, st)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    p = c.params(out)
    ws = torch.empty(max(256, B.spec_beam_select_workspace_size(p)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.spec_beam_select(p, ws)
    for _ in range(2):
        c.scores.copy_(s0), c.lengths.copy_(l0), c.finished.copy_(f0)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


# ------------------------------------------------------------------------------------ reorder
class Reorder:
    def __init__(self, lens, parent, H=2, d=64, bs=16, L=2, dtype=BF16, seed=0, width=None):
        rng = np.random.default_rng(seed)
        self.B, self.W, self.bs, self.lens, self.parent = len(lens), len(parent[0]), bs, lens, parent
        n = width or max(max(lens), 0) // bs + 3
        self.nb = self.B * self.W * n + 5
        self.table = torch.from_numpy(rng.permutation(self.nb)[:self.B * self.W * n].reshape(self.B * self.W, n).astype(np.int32)).cuda()
        shape = (L, self.nb, H, bs, d)
        mk = lambda: torch.from_numpy(rng.integers(0, 256, (*shape, torch.empty(0, dtype=dtype).element_size()), dtype=np.uint8)).cuda().view(dtype).reshape(shape)  # noqa: E731
        self.k, self.v = mk(), mk()
        self.ks = self.vs = None
        if dtype == E4M3:
            self.ks, self.vs = [torch.from_numpy(rng.random(shape[:3])).float().cuda() for _ in range(2)]
        self.status = torch.full((self.B,), 77, dtype=torch.int32, device="cuda")

    def params(self):
        self.held = (U.ints(self.lens), U.ints(self.parent))
        return B.beam_reorder_params(self.k, self.v, self.table, *self.held, self.status, self.ks, self.vs)

    def check(self, stream=None):
        bits = lambda t: t.contiguous().view(torch.uint8).cpu().numpy().reshape(*t.shape, -1)  # noqa: E731
        new, copies, status = beam.reorder(self.table.cpu().numpy(), self.lens, self.parent, self.bs, self.nb)
        want = [bits(t) for t in (self.k, self.v)]
        scales = [t.cpu().numpy().copy() for t in (self.ks, self.vs) if t is not None]
        for _, fr, to, rem in copies:
            for w in want:
                w[:, to, :, :rem] = w[:, fr, :, :rem]
            for sc in scales:
                sc[:, to] = sc[:, fr]
        p = self.params()
        ws = torch.full((B.spec_beam_reorder_workspace_size(p),), 0xA5, dtype=torch.uint8, device="cuda")
        B.spec_beam_reorder(p, ws, stream)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(self.table.cpu().numpy(), new)
        for t, w in zip((self.k, self.v), want):
            np.testing.assert_array_equal(bits(t), w)
        for t, w in zip([t for t in (self.ks, self.vs) if t is not None], scales):
            np.testing.assert_array_equal(t.cpu().numpy(), w)
        assert self.status.cpu().tolist() == status
        return copies


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("bs,d,H,L", [(16, 128, 2, 3), (32, 64, 3, 1), (1, 16, 1, 2), (7, 48, 2, 2), (128, 128, 1, 1)])
def test_reorder_shapes(bs, d, H, L, dtype):
    rng = np.random.default_rng(bs)
    assert Reorder([0, 1, bs, 3 * bs - 1, 250, 40], rng.integers(0, 5, (6, 5)).tolist(), H, d, bs, L, dtype).check() or bs == 1


@pytest.mark.parametrize("parent", [[[0]], [[1, 0]], [[0, 0]], [[1, 1]], [[3, 3, 3, 3]], [[3, 2, 1, 0]], [[2, 2, 0, 0]], [list(range(16))], [[15] * 16], [[7, 7, 0, 3] * 4]])
def test_reorder_parents(parent):
    c = Reorder([37], parent)
    copies = c.check()
    assert len(copies) == len(parent[0]) - len(set(parent[0]))
    c.check()                   # again, over what the first one left


def test_reorder_at_page_bounds_copies_nothing():
    assert Reorder([32, 0], [[1, 1, 1], [2, 2, 0]]).check() == []


def test_reorder_refuses_requests_one_by_one():
    c = Reorder([20, 20, 40, 1000, -1, 17], [[0, 3, 1], [0, -1, 1], [2, 2, 1], [0, 0, 0], [0, 0, 0], [1, 1, 1]], width=6)
    c.table[2 * 3, 2] = c.nb                     # request 2: a writing page outside the pool
    c.table[5 * 3, 1] = c.table[5 * 3 + 2, 1]    # request 5: two beams name one page
    assert c.check() == []
    assert c.status.tolist() == [1, 1, 32, 2, 2, 32]
    c = Reorder([20, 21], [[2, 2, 2], [0, 5, 0]])
    assert len(c.check()) == 2 and c.status.tolist() == [0, 1]


def test_reorder_many_requests_and_layers_in_a_graph():
    rng = np.random.default_rng(8)
    c = Reorder(rng.integers(1, 60, 90).tolist(), rng.integers(0, 4, (90, 4)).tolist(), H=1, d=16, L=5)
    c.check(torch.cuda.Stream())
    p = c.params()
    ws = torch.empty(B.spec_beam_reorder_workspace_size(p), dtype=torch.uint8, device="cuda")
    before = (c.table.clone(), c.k.clone())      # random bits: NaN among them
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.spec_beam_reorder(p, ws)
    g.replay()
    torch.cuda.synchronize()
    after = (c.table.clone(), c.k.clone())
    c.table.copy_(before[0]), c.k.copy_(before[1])
    B.spec_beam_reorder(p, ws)
    torch.cuda.synchronize()
    assert torch.equal(c.table, after[0]) and torch.equal(c.k.view(torch.int16), after[1].view(torch.int16))


# ------------------------------------------------------------------------------------ a whole search
def _rotate(x, pos, base=10000.0):
    h = x.shape[-1] // 2
    ang = pos * base ** (-np.arange(h) / h)
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)], -1)


class Toy:
    """One layer with random weights: enough for the beams to depend on everything that they have read."""

    def __init__(self, V, Hq, H, d, seed):
        rng = np.random.default_rng(seed)
        self.V, self.Hq, self.H, self.d, E = V, Hq, H, d, 24
        self.emb = rng.normal(size=(V, E))
        self.wq, self.wk, self.wv = [rng.normal(size=(E, h * d)) / np.sqrt(E) for h in (Hq, H, H)]
        self.wo = rng.normal(size=(Hq * d, V)) * 3 / np.sqrt(Hq * d)

    def logits(self, seq):
        """After the last of the tokens, by plain causal attention in fp64."""
        e = self.emb[seq]
        q = _rotate((e[-1] @ self.wq).reshape(self.Hq, self.d), len(seq) - 1)
        k = np.stack([_rotate((x @ self.wk).reshape(self.H, self.d), i) for i, x in enumerate(e)])
        v = (e @ self.wv).reshape(len(seq), self.H, self.d)
        out = []
        for h in range(self.Hq):
            x = k[:, h * self.H // self.Hq] @ q[h] / np.sqrt(self.d)
            w = np.exp(x - x.max())
            out.append(w @ v[:, h * self.H // self.Hq] / w.sum())
        return np.concatenate(out) @ self.wo


def _search(toy, prompts, W, steps, bs, dtype, eos, alpha):
    n, d, Bn = toy.V, toy.d, len(prompts)
    prompt_len = [len(p) - 1 for p in prompts]
    wide = max(prompt_len) // bs + steps // bs + 3
    rng = np.random.default_rng(5)
    nb = Bn * W * wide
    table = torch.from_numpy(rng.permutation(nb).reshape(Bn * W, wide).astype(np.int32)).cuda()
    k, v = [torch.zeros((1, nb, toy.H, bs, d), dtype=dtype, device="cuda") for _ in range(2)]
    for b, p in enumerate(prompts):            # the prompt enters beam 0's pages
        for i, t in enumerate(p[:-1]):
            page = int(table[b * W, i // bs])
            k[0, page, :, i % bs] = torch.from_numpy(_rotate((toy.emb[t] @ toy.wk).reshape(toy.H, d), i)).to(dtype)
            v[0, page, :, i % bs] = torch.from_numpy((toy.emb[t] @ toy.wv).reshape(toy.H, d)).to(dtype)
    s = BeamSearch(k, v, table, U.ints(prompt_len), W, toy.Hq, n, eos=eos, alpha=alpha)
    s.spread()
    s.tokens.copy_(torch.tensor([[p[-1]] * W for p in prompts]))
    emb, wq, wk, wv, wo = [torch.from_numpy(m).float().cuda() for m in (toy.emb, toy.wq, toy.wk, toy.wv, toy.wo)]
    ld = -(-n // 8) * 8
    q_in = torch.empty((Bn * W, toy.Hq, d), dtype=dtype, device="cuda")
    q, o = torch.empty_like(q_in), torch.empty_like(q_in)
    kn, vn = [torch.empty((Bn * W, toy.H, d), dtype=dtype, device="cuda") for _ in range(2)]
    logits = torch.zeros((Bn * W, ld), device="cuda")

    def step():
        e = emb[s.tokens.view(-1).long()]
        q_in.copy_((e @ wq).view(q_in.shape))
        kn.copy_((e @ wk).view(kn.shape))
        vn.copy_((e @ wv).view(vn.shape))
        s.write(0, q_in, q, kn, vn)
        s.attention(0, q, o)
        logits[:, :n] = o.view(Bn * W, -1).float() @ wo
        s.advance(logits)

    seqs = [[list(p) for _ in range(W)] for p in prompts]
    for _ in range(steps):
        step()
        par, tok = s.parent.tolist(), s.tokens.tolist()
        seqs = [[list(seqs[b][par[b][j]]) + [tok[b][j]] for j in range(W)] for b in range(Bn)]
    assert s.status.tolist() == [0] * (Bn * W) and s.beam_status.tolist() == [0] * Bn
    return s, seqs, step


@pytest.mark.parametrize("alpha,eos", [(0.0, -1), (0.7, 3)])
def test_search_equals_search_without_a_cache(alpha, eos):
    """fp32 throughout on the device, fp64 over whole sequences on the host: the same beams, with scores to 1e-4
    (steps x logits of size 10 formed in fp32)."""
    W, steps = 4, 11
    toy = Toy(61, 4, 2, 32, 1)
    rng = np.random.default_rng(2)
    prompts = [rng.integers(0, 61, n).tolist() for n in (1, 9, 17, 30)]
    s, seqs, _ = _search(toy, prompts, W, steps, 4, F32, eos, alpha)
    got = s.scores.cpu().numpy()
    for b, p in enumerate(prompts):
        beams = [(list(p), 0.0, 0, False)] + [(list(p), -np.inf, 0, False)] * (W - 1)
        for _ in range(steps):
            x = np.stack([toy.logits(q) for q, *_ in beams])[None]
            par, tok, sc, ln, fin, _ = beam.select(x, np.array([[q[1] for q in beams]]), np.array([[q[2] for q in beams]]),
                                                   np.array([[q[3] for q in beams]]), 1.0, alpha, eos)
            beams = [(beams[par[0, j]][0] + [int(tok[0, j])], sc[0, j], ln[0, j], bool(fin[0, j])) for j in range(W)]
        for j in range(W):
            assert seqs[b][j] == beams[j][0]
            assert abs(got[b, j] - beams[j][1]) < 1e-4
            assert int(s.lengths[b, j]) == beams[j][2] and bool(s.finished[b, j]) == beams[j][3]


def test_search_in_bf16_runs_and_repeats_from_a_graph():
    toy = Toy(300, 8, 2, 128, 3)
    rng = np.random.default_rng(4)
    prompts = [rng.integers(0, 300, n).tolist() for n in (5, 140, 33)]
    s, seqs, step = _search(toy, prompts, 5, 6, 16, BF16, 7, 1.0)
    state = [s.kv_len, s.prefix, s.scores, s.lengths, s.finished, s.tokens, s.block_table, s.k_cache, s.v_cache]
    before = [t.clone() for t in state]
    step()
    want = [s.parent.clone(), s.tokens.clone(), s.scores.clone(), s.block_table.clone(), s.k_cache.clone()]
    for t, b in zip(state, before):
        t.copy_(b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((s.parent, s.tokens, s.scores, s.block_table, s.k_cache), want):
        assert torch.equal(a, b)


def test_search_over_an_8bit_cache_advances():
    W, bs = 3, 16
    table = U.ints(np.arange(6 * 4).reshape(6, 4).tolist())
    k = torch.randint(0, 120, (2, 24, 2, bs, 32), dtype=torch.uint8, device="cuda")
    v, ks = k.flip(1).contiguous(), torch.rand((2, 24, 2), device="cuda")
    s = BeamSearch(k, v, table, U.ints([20, 33]), W, 4, 100, k_scale=ks, v_scale=ks.clone())
    s.spread()
    x = torch.randn((6, 104), device="cuda")
    for _ in range(4):
        s.advance(x)
    assert s.beam_status.tolist() == [0, 0] and s.kv_len.tolist() == [24, 37]
    assert (s.lengths == 4).all() and torch.isfinite(s.scores).all()
