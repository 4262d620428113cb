"""Pins of the 8-bit cache's oracle: the number format against all 256 codes, the scale rule at
its edges, and append / compaction on hand-made examples."""
import numpy as np
import pytest
import torch

from oracle import kv8 as K


def test_rounding_is_the_nearest_code_with_ties_to_even():
    vals = K.e4m3_values()
    codes = np.arange(256)
    fin = ~np.isnan(vals) & (codes < 128)
    pos, even = vals[fin], (codes[fin] % 2 == 0)
    rng = np.random.default_rng(0)
    mids = (pos[1:] + pos[:-1]) / 2
    xs = np.concatenate([pos, mids, np.nextafter(mids, 0), np.nextafter(mids, 1e9), rng.uniform(0, 500, 500),
                         2.0 ** rng.uniform(-14, 9, 500)])
    for x in xs:
        d = np.abs(pos - min(x, 448.0))
        best = np.flatnonzero(d == d.min())
        want = pos[best[0]] if len(best) == 1 else pos[best[even[best]][0]]
        assert K.round_e4m3(x) == want and K.round_e4m3(-x) == -want


def test_rounding_matches_the_library_type():
    x = (torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 60).clamp(-448, 448)
    np.testing.assert_array_equal(x.to(torch.float8_e4m3fn).double().numpy(), K.round_e4m3(x.numpy()))
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    np.testing.assert_array_equal(codes.double().numpy(), K.e4m3_values())


def test_saturation_and_nan():
    np.testing.assert_array_equal(K.round_e4m3([np.inf, -np.inf, 464.0, 1e30]), [448, -448, 448, 448])
    assert np.isnan(K.round_e4m3(np.nan))


@pytest.mark.parametrize("a,s", [(448.0, 1.0), (448.0000001, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                 (1.76, 2.0 ** -7), (0.0, 2.0 ** -100), (1e-45, 2.0 ** -100), (3.4e38, 2.0 ** 119)])
def test_scale_rule(a, s):
    assert K.need_scale(a) == s


def test_append_grows_a_partial_block_and_keeps_its_values():
    codes, scale = np.zeros((2, 1, 4, 2)), np.ones((2, 1))
    K.append(codes, scale, np.array([[[1.0, -2.0]], [[0.5, 0.25]]]), [[1]], [0], [0, 2], 4)
    assert scale[1, 0] == 2.0 ** -7
    np.testing.assert_array_equal(codes[1, 0, :2] * scale[1, 0], [[1, -2], [0.5, 0.25]])
    K.append(codes, scale, np.array([[[900.0, 0.0]]]), [[1]], [2], [0, 1], 4)
    assert scale[1, 0] == 4.0                    # 900 <= 448 * 4
    np.testing.assert_array_equal(codes[1, 0, :3] * scale[1, 0], [[1, -2], [0.5, 0.25], [896, 0]])


def test_append_to_a_fresh_block_ignores_its_stale_scale():
    codes, scale = np.full((1, 1, 4, 2), 7.0), np.full((1, 1), 1e6)
    K.append(codes, scale, np.array([[[1.0, 1.0]]]), [[0]], [0], [0, 1], 4)
    assert scale[0, 0] == 2.0 ** -8 and (codes[0, 0, 0] == 256).all() and (codes[0, 0, 1:] == 7).all()


def test_compact_takes_the_largest_scale_and_keeps_values():
    # block 0 holds one live row and tree rows 0..2, block 1 tree rows 3..6; path 0 -> 4
    codes, scale = np.zeros((2, 1, 4, 1)), np.array([[1.0], [8.0]])
    codes[0, 0, :, 0] = [16, 8, 4, 2]
    codes[1, 0, :, 0] = [1, 2, 3, 4]
    K.compact(codes, scale, [[0, 1]], [1], [[0, 4]], [1], 4)
    assert scale[0, 0] == 8.0 and scale[1, 0] == 8.0
    np.testing.assert_array_equal(codes[0, 0, :3, 0] * scale[0, 0], [16, 8, 16])   # live, root, node 4


def test_compact_leaves_an_unmoved_block_alone():
    codes, scale = np.ones((1, 1, 4, 1)) * 3, np.array([[0.3]])
    K.compact(codes, scale, [[0]], [1], [[0, 1]], [1], 4)
    assert scale[0, 0] == 0.3 and (codes == 3).all()


def test_attention_of_a_row_that_sees_nothing():
    z = np.zeros((1, 1, 4, 2))
    o, lse, *_ = K.tree_attention(np.ones((1, 1, 2)), z, np.ones((1, 1)), z + 1, np.ones((1, 1)), [[0]], [0], [0, 1],
                                  [[False]], 4)
    assert (o == 0).all() and lse[0, 0] == -np.inf


def test_attention_against_dense_softmax():
    rng = np.random.default_rng(2)
    k, v = K.round_e4m3(rng.normal(size=(3, 2, 4, 8)) * 50), K.round_e4m3(rng.normal(size=(3, 2, 4, 8)) * 50)
    ks, vs = 2.0 ** rng.integers(-6, -3, (3, 2)), 2.0 ** rng.integers(-6, -3, (3, 2))
    q = rng.normal(size=(2, 4, 8))
    o, lse, *_ = K.tree_attention(q, k, ks, v, vs, [[2, 0, 1]], [7], [0, 2], [[True, False], [True, True]], 4)
    kf = np.concatenate([k[b] * ks[b][:, None, None] for b in (2, 0, 1)], axis=1)
    vf = np.concatenate([v[b] * vs[b][:, None, None] for b in (2, 0, 1)], axis=1)
    for n, S in ((0, 8), (1, 9)):
        for h in range(4):
            x = torch.tensor(kf[h // 2, :S] @ q[n, h] / np.sqrt(8))
            np.testing.assert_allclose(lse[n, h], torch.logsumexp(x, 0).item(), rtol=1e-12)
            np.testing.assert_allclose(o[n, h], (torch.softmax(x, 0).numpy() @ vf[h // 2, :S]), rtol=1e-10, atol=1e-12)
