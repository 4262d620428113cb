"""GPU tests of the softmax weights that tree attention over the 8-bit cache forms: long flat rests
beside one key that has most of the weight, V scales that lie far apart, blocks of zeros.

Bars, by arithmetic, elementwise.  A weight is rounded to fp16 (2^-11 of itself) and, in units of at
most 16 query rows, split in three e5m2 pieces that leave 2^-10 of it, or 2^-17 of a range in which the
row's largest weight (times its V scale) is at least 2^13: 2^-30 of that, and twice that at most where
a unit is joined of two references.  Longer units: fp16 alone, whose smallest half step is 2^-25 of a
range in which the largest is at least 2^5, 2^-30 as well.  Scores: bf16 queries as two
e4m3 pieces, off by 2^-17.8 max|q| an element, sums in fp32 (2^-17 of their magnitudes), exponents up to
2^7 in fp32 and exp2 (2^-16 together).  Output: one rounding to bf16 (2^-8).
fp32 queries: fp32 products and sums, 2^-17 of the mean absolute value beside the scores' error.
Over all outputs the roundings to bf16 are independent: their root mean square is at most
2^-8 / sqrt(3) of the outputs', which with the weights' 2^-10 + 2^-11 added in squares is below 2.8e-3.
(kv8_util.check_attention's bars are wider: they allow for weights in e4m3 pieces.)"""
import numpy as np
import pytest
import torch

import kv8_util as U
from oracle import kv8 as K

pytestmark = pytest.mark.gpu


def fill(c, r, kf, vf):
    """Request r's slots take the rows kf, vf [slots, H, d], each page's scale the smallest that holds them."""
    bs, S, H = c.bs, kf.shape[0], kf.shape[1]
    n = -(-S // bs)
    pages = torch.from_numpy(c.table_np[r][:n].astype(np.int64)).cuda()
    for codes, scale, x in ((c.k, c.ks, kf), (c.v, c.vs, vf)):
        rows = np.zeros((n * bs, H, c.d))
        rows[:S] = x
        rows = rows.reshape(n, bs, H, c.d).transpose(0, 2, 1, 3)
        a = np.abs(rows).max(axis=(2, 3))
        s = np.ones_like(a)
        s.flat = [K.need_scale(float(v)) for v in a.flat]
        q = torch.from_numpy(K.round_e4m3(rows / s[:, :, None, None])).to(U.E4M3).view(torch.uint8)
        if S % bs:                                  # the last page's other rows stay poisoned
            q[-1, :, S % bs:] = 0x7F
        codes.view(torch.uint8)[pages] = q.cuda()
        scale[pages] = torch.from_numpy(s).float().cuda()


def check(c):
    """Compares c.o and c.lse with the definition in 64 bits; returns that O."""
    d, H, Hq = c.d, c.ks.shape[1], c.q.shape[1]
    G = Hq // H
    f32 = c.q.dtype == torch.float32
    pieces, left = 2.0 ** -10 if c.T_max * G <= 16 else 0.0, 2 * 2.0 ** -30
    kc, vc = (torch.nan_to_num(t.double()).cpu() for t in (c.k, c.v))
    ks, vs, cq, co, cl = (t.double().cpu() for t in (c.ks, c.vs, c.q, c.o, c.lse))
    outs = []
    for r, (P, T) in enumerate(zip(c.prefix, c.sizes)):
        n0, S = int(c.off_np[r]), P + T
        ids = torch.from_numpy(c.table_np[r][:-(-S // c.bs)].astype(np.int64))
        seen = torch.ones((T, S), dtype=torch.bool)
        for i in range(T):
            seen[i, P:] = torch.tensor([bool((c.bits[n0 + i] >> j) & 1) for j in range(T)])
        seen = seen[:, None, :].expand(T, G, S).reshape(T * G, S)
        for h in range(H):
            k = (kc[ids, h] * ks[ids, h][:, None, None]).reshape(-1, d)[:S]
            code = vc[ids, h].reshape(-1, d)[:S]
            s = vs[ids, h].repeat_interleave(c.bs)[:S]
            v = code * s[:, None]
            q = cq[n0:n0 + T, h * G:(h + 1) * G].reshape(T * G, d)
            x = (q @ k.T / d ** 0.5).masked_fill(~seen, -np.inf)
            lse = torch.logsumexp(x, 1)
            w = torch.exp(x - lse[:, None])
            o, mass = w @ v, w @ v.abs()
            zero = torch.zeros((), dtype=torch.float64)
            E = 2.0 ** -16 + 2.0 ** -17 * torch.where(seen, q.abs() @ k.abs().T / d ** 0.5, zero).amax(1)
            if not f32:
                E += 2.0 ** -17.8 * q.abs().amax(1) / d ** 0.5 * torch.where(seen, k.abs().sum(1)[None], zero).amax(1)
            rest = (w * s).amax(1)[:, None] * (seen.double() @ code.abs())
            if f32:
                tol = (2 * E[:, None] + 2.0 ** -17) * mass
            else:
                tol = (2 * E[:, None] + pieces + 2.0 ** -11) * mass + left * rest + 2.0 ** -8 * o.abs()
            go = co[n0:n0 + T, h * G:(h + 1) * G].reshape(T * G, d)
            gl = cl[n0:n0 + T, h * G:(h + 1) * G].reshape(T * G)
            worst = ((go - o).abs() / (tol + 1e-30)).max().item()
            assert worst <= 1, worst
            assert ((gl - lse).abs() <= E + 2.0 ** -21 * lse.abs() + 2.0 ** -19).all()
            outs.append((o, go))
    o, go = (torch.cat([x[i] for x in outs]) for i in (0, 1))
    assert torch.linalg.norm(go - o) <= (2e-5 if f32 else 2.8e-3) * torch.linalg.norm(o)
    return o


FORMS = [(4, 1, 1, torch.bfloat16), (2, 2, 7, torch.bfloat16), (4, 1, 4, torch.bfloat16),
         (4, 1, 20, torch.bfloat16), (2, 1, 80, torch.bfloat16), (2, 1, 2, torch.float32)]


def sink_case(Hq, H, T, dtype, P, at, part, spread, seed):
    """One key at slot `at` with about `part` of the weight and small V, the rest with scores N(0, spread) and
    V of mean 0.7."""
    c = U.AttnCase([P], [T], Hq, H, dtype=dtype, seed=seed)
    rng = np.random.default_rng(seed)
    d, S = c.d, P + T
    base = rng.normal(size=d)
    c.q = torch.from_numpy(base + 0.02 * rng.normal(size=(T, Hq, d))).cuda().to(dtype)
    kf = rng.normal(size=(S, H, d)) * spread * np.sqrt(d) / np.linalg.norm(base)
    kf[at] = base * np.sqrt(d) / (base @ base) * (np.log(part / (1 - part) * S) + spread ** 2 / 2)
    vf = 0.7 + 0.2 * rng.normal(size=(S, H, d))
    vf[at] = 0.01 * rng.normal(size=(H, d))
    fill(c, 0, kf, vf)
    return c


@pytest.mark.parametrize("Hq,H,T,dtype", FORMS)
@pytest.mark.parametrize("P,where,part", [(8000, 0.0, 0.5), (8000, 0.5, 0.9), (32000, 0.0, 0.9), (32000, 0.5, 0.98), (32000, 1.0, 0.7)])
def test_a_long_rest_beside_one_heavy_key(Hq, H, T, dtype, P, where, part):
    c = sink_case(Hq, H, T, dtype, P, min(P - 1, int(P * where)), part, 0.5, seed=int(P * where) + T)
    c.run()
    o = check(c)
    assert 0.7 * (1 - part) / 3 < o.abs().mean().item() < 0.7 * (1 - part) * 3


@pytest.mark.parametrize("Hq,H,T,dtype", FORMS[:-1])
@pytest.mark.parametrize("part", [0.9, 0.999])
def test_an_exactly_flat_rest_beside_one_heavy_key(Hq, H, T, dtype, part):
    """Every weight of the rest is rounded the same way: nothing averages out."""
    c = sink_case(Hq, H, T, dtype, 30000, 77, part, 0.0, seed=T)
    c.run()
    check(c)


@pytest.mark.parametrize("Hq,H,T,dtype", FORMS)
@pytest.mark.parametrize("extra", [8, 12])
def test_blocks_whose_v_scale_is_far_above_the_others(Hq, H, T, dtype, extra):
    """Some blocks need a V scale 2^extra times the others' for a column that the others' rows fill too."""
    P, rng = 4000, np.random.default_rng(extra + T)
    c = U.AttnCase([P], [T], Hq, H, dtype=dtype, seed=T)
    kf = rng.normal(size=(P + T, H, c.d)) * 0.3
    vf = 0.7 + 0.2 * rng.normal(size=(P + T, H, c.d))
    for s in (5, 1000, 2222, 3999):
        vf[s, :, 3] = 2.0 ** extra
    fill(c, 0, kf, vf)
    c.run()
    check(c)


@pytest.mark.parametrize("Hq,H,T,dtype", FORMS)
def test_blocks_of_zeros_in_v_count_in_the_sums(Hq, H, T, dtype):
    """Every other block's V is zero (scale 2^-100 beside scales up to 2^2): half of the weight."""
    P, rng = 3000, np.random.default_rng(T)
    c = U.AttnCase([P], [T], Hq, H, dtype=dtype, seed=T)
    kf = rng.normal(size=(P + T, H, c.d)) * 0.3
    vf = (0.7 + 0.2 * rng.normal(size=(P + T, H, c.d))) * 500
    vf[(np.arange(P + T) // c.bs) % 2 == 0] = 0
    fill(c, 0, kf, vf)
    assert (c.vs == 2.0 ** -100).any() and (c.vs == 2.0).any()
    c.run()
    check(c)


@pytest.mark.parametrize("Hq,H,T,dtype", FORMS)
def test_a_long_cache_of_zero_v_rows(Hq, H, T, dtype):
    """All V scales at 2^-100: the row sums stay finite, O is 0."""
    P, rng = 30000, np.random.default_rng(T)
    c = U.AttnCase([P], [T], Hq, H, dtype=dtype, seed=T)
    fill(c, 0, rng.normal(size=(P + T, H, c.d)) * 0.1, np.zeros((P + T, H, c.d)))
    c.run()
    assert (c.o[:c.N] == 0).all()
    check(c)


@pytest.mark.parametrize("Hq,H,T,dtype,big", [f + (b,) for f in FORMS[:3] + FORMS[-1:] for b in (1e3, 1e12)]
                         + [(16, 8, 1, torch.bfloat16, 1e12), (16, 8, 7, torch.bfloat16, 1e12), (16, 8, 20, torch.bfloat16, 1e3)])
@pytest.mark.parametrize("at", [5, 3000])
def test_pages_of_zeros_beside_one_heavy_key_with_large_v(Hq, H, T, dtype, big, at):
    """The rest is zeros in V (scales of 2^-100) and a third of the weight, the heavy key's V up to `big`;
    with eight KV heads a CTA walks several tiles before that key and after it."""
    P = 20000 if H < 8 else 6000
    c = sink_case(Hq, H, T, dtype, P, at, 0.67, 0.3, seed=T)
    rng = np.random.default_rng(T)
    ids, S = c.table_np[0][:-(-(P + T) // c.bs)], P + T
    kf = np.nan_to_num(U.values(c.k)[ids]) * c.ks.double().cpu().numpy()[ids][:, :, None, None]
    vf = np.zeros((S, H, c.d))
    vf[at] = big * rng.uniform(0.2, 1.0, (H, c.d))
    fill(c, 0, kf.transpose(0, 2, 1, 3).reshape(-1, H, c.d)[:S], vf)
    c.run()
    o = check(c)
    assert o.abs().mean() < 0.8 * np.abs(vf[at]).mean()
