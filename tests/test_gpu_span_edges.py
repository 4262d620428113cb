"""Windowed and shared-prefix attention at their edges: masks with bits behind the tree, scores of any finite size,
values that are not finite under weights that underflow, and group arrays that cannot be."""
import numpy as np
import pytest
import torch

import kv8_util as U
import span_util as S
from oracle import span

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# Which kernel a call takes: at most 16 query rows a request and head, more of them (one row tile, two), fp32.
KERNELS = {"rows": dict(dtype=BF16, T=2, Hq=8, H=2), "tile": dict(dtype=BF16, T=20, Hq=8, H=2), "pairs": dict(dtype=BF16, T=64, Hq=8, H=2),
           "cores": dict(dtype=F32, T=5, Hq=4, H=2)}


# ------------------------------------------------------------------------------------ masks
@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("sizes,T_max,G,dtype", [([1, 3, 5], 8, 2, BF16), ([5, 33, 70], 100, 4, BF16), ([5, 33, 70], 100, 4, F32), ([31, 32, 64], 256, 1, BF16),
                                                 ([2, 40, 9], 64, 2, F32)])
def test_mask_bits_behind_the_tree_do_not_count(kind, sizes, T_max, G, dtype):
    """Neither for what a node sees nor for its depth."""
    rng = np.random.default_rng(T_max)
    room = 32 * ((T_max + 31) // 32)
    bits = []
    for t in sizes:
        for i, b in enumerate(U.chain_bits(t) if t < 40 else U.tree_bits(t, rng)):
            stray = sum(1 << int(p) for p in rng.choice(np.arange(t, room), min(room - t, 1 + i % 9), replace=False))
            bits.append(b | stray)
    kw = dict(window=23, sinks=3) if kind == "window" else dict(groups=[(0, 2, 40), (2, 3, 7)])
    c = S.Case([300, 45, 7], sizes, Hq=2 * G, H=2, dtype=dtype, T_max=T_max, bits=bits, seed=40, **kw)
    c.run()
    S.check(c)


# ------------------------------------------------------------------------------------ large scores
def _scores(c):
    """(row, query head, its scores in 64 bits, their products' magnitudes, the slots' values) of every row that sees
    something."""
    G = c.q.shape[1] // c.k.shape[1]
    q, table = c.q.double().cpu().numpy(), torch.from_numpy(c.table_np).long()
    for r, (P, T) in enumerate(zip(c.prefix, c.sizes)):
        first, length = r, 0
        for a, b, ln in c.groups or []:
            if a <= r < b:
                first, length = a, ln
        slots = torch.arange(P + T)
        page = torch.where(slots < length, table[first][torch.clamp(slots // c.bs, max=table.shape[1] - 1)], table[r][slots // c.bs])
        at = (page.clamp(min=0).cuda(), slice(None), (slots % c.bs).cuda())
        K, V = [t[at[0], :, at[2]].double().cpu().numpy() for t in (c.k, c.v)]
        for i in range(T):
            n = int(c.off_np[r]) + i
            seen = np.array(span.visible(c.bits[n], P, T, c.window, c.sinks), dtype=int)
            for h in range(c.q.shape[1] if len(seen) else 0):
                k, x = K[seen, h // G], q[n, h] / np.sqrt(q.shape[2])
                yield n, h, k @ x, np.abs(k) @ np.abs(x), V[seen, h // G]


def _one_hot(c):
    """Rows whose best score stands out of what fp32 sums and one rounding of a score can move (2^-17 of the products'
    magnitudes for each, 64 for an exponential that is nothing beside it): the output is that key's V, rounded
    once (pair units round its weight before), and the log-sum-exp that score.  Returns how many there are."""
    o, lse = c.o[:c.N].double().cpu().numpy(), c.lse[:c.N].double().cpu().numpy()
    found = 0
    for n, h, x, size, V in _scores(c):
        at = int(np.argmax(x))
        slack = 2.0 ** -17 * size.max()
        rest = np.delete(x, at)
        if len(rest) and x[at] - rest.max() < 2 * slack + 64:
            continue
        found += 1
        assert (np.abs(o[n, h] - V[at]) <= 2.0 ** -7 * np.abs(V[at])).all(), (n, h)
        assert abs(lse[n, h] - x[at]) <= slack + 2.0 ** -20 * abs(x[at]), (n, h)
    return found


def _large(kernel, kind, exps, sign, seed, prefix=(700, 90, 0, 1400), T=None):
    k = KERNELS[kernel]
    T = T or k["T"]
    kw = dict(window=5000, sinks=2) if kind == "window" else dict(groups=[(0, 2, 90), (2, 4, 0)])
    c = S.Case(list(prefix), [T] * len(prefix), Hq=k["Hq"], H=k["H"], dtype=k["dtype"], seed=seed, **kw)
    if sign < 0:            # every score negative
        c.k.copy_(c.k.abs())
        c.q.copy_(-c.q.abs())
    step = torch.tensor([float(exps[n % len(exps)]) for n in range(c.q.shape[0])], device="cuda")
    c.q.copy_(c.q.float() * torch.exp2(step)[:, None, None])
    c.run()
    return c


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exps", [(26,), (27, 28, 29), (30, 31), (33, 40), (60, 90), (0, 30, 5, 100)], ids=str)
def test_finite_scores_of_any_size_under_a_window(kernel, exps, sign):
    """A score of 2^30 and more is a rounded number whose last place is tens of units of the exponent."""
    c = _large(kernel, "window", exps, sign, 41)
    S.check(c)
    assert _one_hot(c) > 0.5 * c.N * c.q.shape[1] * (1 - exps.count(0) / len(exps))


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("exps", [(26,), (30, 31), (33, 40), (0, 30, 5, 100)], ids=str)
def test_finite_scores_of_any_size_under_a_shared_prefix(kernel, exps, sign):
    c = _large(kernel, "shared", exps, sign, 42)
    S.check(c)
    assert _one_hot(c) > 0.5 * c.N * c.q.shape[1] * (1 - exps.count(0) / len(exps))


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_large_scores_of_equal_keys(kernel):
    """The best key stands in many slots of a unit: each of them has the same weight.  (Units that are not cut, of one key tile
    but for the rows kernel's: a piece's log-sum-exp is one fp32 number, which at 2^36 does not say how many keys it
    came from.)"""
    k = KERNELS[kernel]
    prefix = {"rows": [250, 120], "tile": [100, 60], "pairs": [50, 60], "cores": [50, 40]}[kernel]
    c = S.Case(prefix, [k["T"]] * 2, Hq=k["Hq"], H=k["H"], dtype=k["dtype"], window=20000, seed=43)
    u = torch.randn((128,), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    c.q.copy_((u * 2.0 ** 33).expand_as(c.q))
    live = ~c.k.isnan()
    keys = torch.where((torch.arange(c.k.shape[2], device="cuda") % 2 == 0)[:, None], u, -u).expand_as(c.k).to(c.k.dtype)
    c.k.copy_(torch.where(live, keys, c.k))
    c.run()
    o, lse = c.o.double().cpu().numpy(), c.lse.double().cpu().numpy()
    for n, h, x, size, V in _scores(c):
        best = x.max() - x <= 1e-12 * np.abs(x).max()
        assert best.sum() >= 20
        want, mass = V[best].mean(axis=0), np.abs(V[best]).mean(axis=0)
        # weights of 1, whose sum and products are exact in any order up to fp32's 2^-24 for each of 150 terms
        assert (np.abs(o[n, h] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -11 * mass).all(), (n, h)
        assert abs(lse[n, h] - x.max()) <= 2.0 ** -17 * size.max()


# ------------------------------------------------------------------------------------ not finite, and far away
@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("far,length", [(128, 250), (128, 380), (128, 640), (4600, 9000), (6000, 6200)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_value_that_is_not_finite_shows_under_any_weight(kernel, kind, far, length, value):
    """Slots below `far` have scores some 600 below the others', so that the weights of their tiles, of the slot or
    the group of tiles that they are in, or of whole pieces are 0 in fp32; one of them has a bad V."""
    k = KERNELS[kernel]
    T = k["T"]
    kw = dict(window=20000) if kind == "window" else dict(groups=[(0, 2, far)])
    prefix = [length, length + 9]
    c = S.Case(prefix, [T] * 2, Hq=k["Hq"], H=k["H"], dtype=k["dtype"], seed=44, **kw)
    u = torch.randn((128,), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    c.q.copy_(c.q.float() * 0.3 + u)
    slot = far // 2 + 3
    for r in range(2):
        ids = torch.from_numpy(c.table_np[r]).long().cuda()
        low = torch.arange(ids.numel() * c.bs, device="cuda").view(-1, c.bs) < far
        for p in range(ids.numel()):
            if ids[p] >= 0:
                c.k[ids[p]] = torch.where(low[p][None, :, None], (-60 * u).to(c.k.dtype), c.k[ids[p]])
    c.run()
    S.check(c)
    hit = c.table_np[0, slot // c.bs]
    c.v[int(hit), 1, slot % c.bs, 5] = value
    before = c.o.clone()
    c.run()
    rows = c.N if kind == "shared" else T       # who sees the slot
    G = c.q.shape[1] // 2
    assert (~torch.isfinite(c.o[:rows, G:, 5])).all()
    assert torch.equal(c.o[:, :G], before[:, :G]) and torch.equal(c.o[rows:], before[rows:])


# ------------------------------------------------------------------------------------ groups that cannot be
GROUPS = [(0, 2, 30), (2, 4, 50), (4, 6, 10)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offsets", [[0, 4, 2, 6], [0, 6, 6, 2], [3, 2, 4, 6], [0, 2, 1, 6], [6, 4, 2, 0]])
def test_group_offsets_that_go_backwards(dtype, offsets):
    """Groups would overlap: no request can be told which is its own, and no row is written."""
    c = S.Case([60, 61, 90, 95, 40, 41], [1, 2, 1, 1, 2, 1], Hq=4, H=2, groups=GROUPS, dtype=dtype, seed=45)
    c.group_off.copy_(torch.tensor(offsets))
    c.run()
    assert c.status.tolist() == [2] * 6
    assert (c.o == 77).all() and (c.lse == 55).all()


def test_group_offsets_that_go_backwards_among_many():
    n = 1300
    c = S.Case([9] * n, [1] * n, Hq=2, H=1, groups=[(i, i + 2, 5) for i in range(0, n, 2)], seed=46)
    c.group_off[600] = 1205
    c.run()
    assert c.status.tolist() == [2] * n and (c.o == 77).all()


def test_groups_without_requests():
    c = S.Case([60, 61, 90, 95], [1, 2, 1, 1], Hq=4, H=2, groups=[(0, 2, 30), (2, 4, 50)], seed=47)
    c.group_off, c.shared = U.ints([0, 0, 2, 4, 4]), U.ints([1000, 30, 50, -3])
    c.run()
    S.check(c)
    assert c.status.tolist() == [0] * 4


@pytest.mark.parametrize("length", [(1 << 31) - 1, (1 << 31) - 8, (1 << 31) - 1024, 1 << 30])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_shared_length_at_the_end_of_32_bits(dtype, length):
    c = S.Case([60, 61, 90, 95], [1, 2, 1, 1], Hq=4, H=2, groups=[(0, 2, 30), (2, 4, 50)], dtype=dtype, seed=48)
    c.shared[1] = length
    c.run()
    assert c.status.tolist() == [0, 0, 2, 2]
    S.check(c, rows=[0, 1, 2])
    assert (c.o[3:] == 77).all()


# ------------------------------------------------------------------------------------ what roundings there are
@pytest.mark.parametrize("kind,T,n", [("window", 1, 5), ("window", 4, 5), ("window", 7, 3), ("window", 8, 200), ("shared", 1, 200), ("shared", 5, 3)])
def test_weights_of_few_rowed_units_keep_two_pieces(kind, T, n):
    """Units of one row tile hold a weight as two bf16 pieces (2^-16 of it), so that the output's own rounding is all that
    is seen: the root mean square of the error is within a tenth of what rounding the exact output gives.  One piece
    (2^-8 / sqrt(3) of a weight at most) would add a third of it, as it does in pair units (0.0022 for 0.0017)."""
    rng = np.random.default_rng(T + n)
    prefix = [100 + int(x) for x in rng.integers(0, 200, n)]
    kw = dict(window=90) if kind == "window" else dict(groups=[(0, 2, 100), (2, n, 0)])
    c = S.Case(prefix, [T] * n, Hq=8, H=2, q_scale=0.1, seed=49, **kw)
    c.run()
    o, _ = S.check(c)
    once = torch.from_numpy(o).to(BF16).double().numpy()
    err = np.linalg.norm(c.o[:c.N].double().cpu().numpy() - o)
    assert err <= 1.1 * np.linalg.norm(once - o)
