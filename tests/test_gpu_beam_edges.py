"""Beam selection at small temperatures and large logits, its length penalty's precision, and searches one after
another on one BeamSearch."""
import numpy as np
import pytest
import torch

import kv8_util as U
from test_gpu_beam import Select, Toy, _rotate
from speculative_decoding_draft_tree_gb300.api import BeamSearch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
LOWEST = {F32: float(np.finfo(np.float32).min), BF16: float(torch.finfo(BF16).min)}


# ------------------------------------------------------------------------------------ sharp rows
def _near_choices(c, floor=-1e4):
    """The choices whose scores the oracle has above `floor` (what lies below is a logit that is not its row's
    largest, divided by a tiny temperature): same beams and tokens, scores to 1e-5 (a sum of a few weights of 1,
    one rounding).  No beam is finished, no length counts."""
    x = c.rows[:, :c.V].double().cpu().numpy().reshape(c.B, c.W, c.V) / c.tau
    m = x.max(axis=2, keepdims=True)
    total = c.scores.double().cpu().numpy()[:, :, None] + (x - m) - np.log(np.exp(x - m).sum(axis=2, keepdims=True))
    total = total.reshape(c.B, -1)
    order = np.argsort(-total, axis=1, kind="stable")[:, :c.W]
    want = np.take_along_axis(total, order, 1)
    got = c.run()
    near = want > floor
    np.testing.assert_array_equal(got[0][near], (order // c.V)[near])
    np.testing.assert_array_equal(got[1][near], (order % c.V)[near])
    assert (np.abs(got[2] - want)[near] <= 1e-5 * (1 + np.abs(want[near]))).all()
    return near


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0.0, 1000.0, -1000.0])
@pytest.mark.parametrize("tau", [1e-6, 1e-8, 1e-9, 1e-12, 1e-30])
@pytest.mark.parametrize("W,V", [(1, 300), (3, 5000), (4, 152064)])
def test_tiny_temperatures_take_each_rows_largest(W, V, tau, offset, dtype):
    """Logits over tau beyond what fp32 tells apart in whole numbers, of both signs."""
    rng = np.random.default_rng(V)
    x = rng.normal(size=(3, W, V)) * 3 + offset
    s = -rng.random((3, W))
    c = Select(x, s, rng.integers(1, 50, (3, W)), np.zeros((3, W)), V, tau=tau, eos=2, dtype=dtype)
    assert _near_choices(c).sum() >= 3 * W          # each beam's largest token at least


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [40, 3000, 100000])
@pytest.mark.parametrize("big", [25.0, -25.0])
def test_tiny_temperatures_count_equal_logits(V, dtype, big):
    """Several tokens tie for the largest logit, in one segment of the row and over all; the one next to it in the type's
    order does not join them."""
    step = 2.0 ** (-7 if dtype == BF16 else -23) * 16
    x = np.full((1, 2, V), big - 3 * step)
    x[0, 0, [3, V // 2, V - 1]] = big
    x[0, 1, [0, V - 2]] = big
    x[0, 1, 7] = big - step
    c = Select(x, np.array([[-0.25, -0.5]]), np.full((1, 2), 3), np.zeros((1, 2)), V, tau=1e-9, dtype=dtype)
    assert _near_choices(c).all()
    got = c.run()                   # -0.25 - ln 3 = -1.35 lies below -0.5 - ln 2
    np.testing.assert_allclose(got[2][0], [-0.5 - np.log(2)] * 2, atol=1e-6)
    assert got[0].tolist() == [[1, 1]] and got[1].tolist() == [[0, V - 2]]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tau", [1.0, 0.5, 1e-9])
def test_logits_of_the_types_lowest_value(dtype, tau):
    """As masks: they weigh nothing beside others; a row of nothing else is a uniform one."""
    V = 700
    x = np.full((2, 2, V), LOWEST[dtype])
    x[0, 0, [5, 6]] = 1.5
    x[0, 1, 9] = -2.0
    c = Select(x, np.array([[-1.0, -0.5], [-1.0, -3.0]]), np.full((2, 2), 3), np.zeros((2, 2)), V, tau=tau, dtype=dtype)
    got = c.run()
    assert got[0][0].tolist() == [1, 0] and got[1][0].tolist() == [9, 5]
    np.testing.assert_allclose(got[2][0], [-0.5, -1 - np.log(2)], atol=1e-6)
    assert got[0][1].tolist() == [0, 0] and got[1][1].tolist() == [0, 1]
    np.testing.assert_allclose(got[2][1], [-1 - np.log(V)] * 2, atol=1e-5)


def test_a_nan_or_an_infinity_takes_a_sharp_row_out():
    V = 3000
    for bad in (np.nan, np.inf):
        x = np.random.default_rng(1).normal(size=(1, 3, V)) + 40
        x[0, 1, 1234] = bad
        got = Select(x, np.array([[-2.0, 0.0, -1.0]]), np.full((1, 3), 3), np.zeros((1, 3)), V, tau=1e-10).run()
        assert got[0][0].tolist()[:2] == [2, 0] and (got[0][0] != 1).all()


def test_the_length_penalty_tells_ranks_a_few_parts_in_1e9_apart():
    """Ranks of finished beams are score / ((5 + length) / 6)^alpha with nothing else rounded: log2 and the power are
    within 1.6e-9 x alpha x ln 2 and 1.2e-9, so that two ranks that lie 6e-9 apart come in their order."""
    rng = np.random.default_rng(3)
    scores, lengths, order = [], [], []
    alpha = 0.7
    while len(scores) < 400:
        n = rng.integers(1, 4000, 2)
        pen = ((5.0 + n) / 6.0) ** alpha
        s = np.float32(-rng.random() * 50 - 1)
        t = np.float32(float(s) / pen[0] * pen[1])
        r = np.array([float(s), float(t)]) / pen
        gap = abs(r[0] / r[1] - 1)
        if 6e-9 < gap < 2e-8:
            scores.append([s, t])
            lengths.append(n.tolist())
            order.append([0, 1] if r[0] > r[1] else [1, 0])
    c = Select(np.zeros((400, 2, 8)), np.array(scores), lengths, np.ones((400, 2)), 8, alpha=alpha, eos=3)
    assert c.run()[0].tolist() == order


# ------------------------------------------------------------------------------------ several searches
class _Searches:
    """A BeamSearch over one toy model's fp32 cache, and what a search gives: beams' tokens and scores."""

    def __init__(self, prompts, W, room, bs=4):
        self.toy, self.W, self.bs = Toy(61, 4, 2, 32, 1), W, bs
        n = len(prompts)
        wide = max(len(p) - 1 for p in prompts) // bs + room
        nb = n * W * wide
        self.table = torch.from_numpy(np.random.default_rng(5).permutation(nb).reshape(n * W, wide).astype(np.int32)).cuda()
        self.k, self.v = [torch.zeros((1, nb, 2, bs, 32), device="cuda") for _ in range(2)]
        self.prompt_len = U.ints([len(p) - 1 for p in prompts])
        self.s = BeamSearch(self.k, self.v, self.table, self.prompt_len, W, 4, 61, eos=3, alpha=0.6)
        t = self.toy
        self.emb, self.wq, self.wk, self.wv, self.wo = [torch.from_numpy(m).float().cuda() for m in (t.emb, t.wq, t.wk, t.wv, t.wo)]
        self.put(prompts)

    def put(self, prompts):
        """The prompts enter the pages of each request's beam 0."""
        self.prompts = prompts
        table, t = self.table.cpu().numpy(), self.toy
        for b, p in enumerate(prompts):
            for i, x in enumerate(p[:-1]):
                page = int(table[b * self.W, i // self.bs])
                self.k[0, page, :, i % self.bs] = torch.from_numpy(_rotate((t.emb[x] @ t.wk).reshape(2, 32), i)).float()
                self.v[0, page, :, i % self.bs] = torch.from_numpy((t.emb[x] @ t.wv).reshape(2, 32)).float()

    def search(self, steps):
        s, W, n = self.s, self.W, len(self.prompts)
        s.spread()
        s.tokens.copy_(torch.tensor([[p[-1]] * W for p in self.prompts]))
        q, o = [torch.empty((n * W, 4, 32), device="cuda") for _ in range(2)]
        logits = torch.zeros((n * W, 64), device="cuda")
        seqs = [[[] for _ in range(W)] for _ in range(n)]
        for _ in range(steps):
            e = self.emb[s.tokens.view(-1).long()]
            s.write(0, (e @ self.wq).view(-1, 4, 32), q, (e @ self.wk).view(-1, 2, 32), (e @ self.wv).view(-1, 2, 32))
            s.attention(0, q, o)
            logits[:, :61] = o.view(n * W, -1) @ self.wo
            s.advance(logits)
            par, tok = s.parent.tolist(), s.tokens.tolist()
            seqs = [[seqs[b][par[b][j]] + [tok[b][j]] for j in range(W)] for b in range(n)]
        torch.cuda.synchronize()
        return seqs, s.scores.clone(), s.lengths.clone()

    def clean(self):
        return (self.s.status == 0).all().item() and (self.s.beam_status == 0).all().item()


PROMPTS = [[5, 9, 1, 30, 44, 2, 17], [8, 8, 60], [3] * 13]


def _same(a, b):
    return a[0] == b[0] and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_a_second_search_is_the_first_again():
    """The first one fills pages, so that beams name one in common; the second starts from the prompts."""
    c = _Searches(PROMPTS, 4, 5)
    first = c.search(11)
    assert c.clean()
    c.s.begin()
    again = c.search(11)
    assert c.clean() and _same(first, again)


def test_a_search_after_one_that_ran_out_of_its_table():
    c = _Searches(PROMPTS, 4, 3)
    first = c.search(6)
    c.s.begin()
    c.search(18)                    # past the longest prompt's table row
    assert not c.clean()
    c.s.begin()
    again = c.search(6)
    assert c.clean() and _same(first, again)


def test_other_prompts_by_another_table():
    other = [[7, 50, 2, 2, 9], [1, 2, 3, 4, 5, 6, 7, 8, 9, 10], [33, 12]]
    fresh = _Searches(other, 4, 6)
    want = fresh.search(9)
    c = _Searches(PROMPTS, 4, 5)
    c.search(11)
    table = torch.from_numpy(np.random.default_rng(9).permutation(c.k.shape[1]).reshape(c.table.shape).astype(np.int32)).cuda()
    c.prompt_len.copy_(U.ints([len(p) - 1 for p in other]))
    for _ in range(2):              # and again, from the table that was given last
        c.s.begin(table)
        table = None
        c.put(other)
        got = c.search(9)
        assert c.clean() and got[0] == want[0]
        torch.testing.assert_close(got[1], want[1], atol=1e-4, rtol=0)


def test_begin_refuses_another_tables_shape():
    c = _Searches(PROMPTS, 4, 5)
    with pytest.raises(ValueError, match="block_table"):
        c.s.begin(c.table[:, :-1].contiguous())
    with pytest.raises(ValueError):
        c.s.begin(c.table.long())
