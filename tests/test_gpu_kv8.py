"""GPU parity of the 8-bit cache's operators (append, tree attention, compaction, fork) with the
fp64 oracle.  Codes, scales, tables and lengths are compared bit for bit: every quantisation is one
division by (or product with) an fp32 number and one rounding to e4m3.  Attention's bars are in
kv8_util.check_attention."""
import numpy as np
import pytest
import torch

import kv8_util as U
from oracle import kv8 as K
from speculative_decoding_draft_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
E4M3 = U.E4M3


# ------------------------------------------------------------------------------------ append
class AppendCase:
    def __init__(self, start, sizes, H=2, d=128, bs=16, dtype=torch.bfloat16, seed=0, pad=0, fused=False, width=None, extra=3):
        rng = np.random.default_rng(seed)
        need = [-(-(max(p, 0) + t) // bs) for p, t in zip(start, sizes)]
        self.nb = sum(need) + extra
        self.table_np = U.table_for(need, self.nb, rng, width)
        (self.k, self.ks), (self.v, self.vs) = [tuple(t[0] for t in U.random_cache(1, self.nb, H, bs, d, rng)) for _ in range(2)]
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
        self.N = int(off[-1]) + pad
        g = torch.Generator(device="cuda").manual_seed(seed)
        mag = torch.exp2(torch.rand((self.N, H, 1), generator=g, device="cuda") * 8 - 4)
        x = lambda: (torch.randn((self.N, H, d), generator=g, device="cuda") * mag).to(dtype)  # noqa: E731
        if fused:    # slices of a fused projection: q heads, k heads, v heads of each token
            qkv = torch.zeros((self.N, 3 * H + 2 * H, d), dtype=dtype, device="cuda")
            qkv[:, 3 * H:4 * H], qkv[:, 4 * H:] = x(), x()
            self.k_new, self.v_new = qkv[:, 3 * H:4 * H], qkv[:, 4 * H:]
        else:
            self.k_new, self.v_new = x(), x()
        self.start, self.off, self.bs = start, off, bs
        self.table = torch.from_numpy(self.table_np).cuda()
        self.status = torch.zeros(len(start), dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        self.held = (U.ints(self.start), U.ints(self.off.tolist()))
        p = B.kv8_append_params(self.k_new, self.v_new, self.k, self.v, self.ks, self.vs, self.table, *self.held, self.status)
        B.spec_kv8_append(p, stream)
        torch.cuda.synchronize()

    def check(self):
        st0 = self.status.cpu().numpy().copy()
        want = []
        for codes, scale, x in ((self.k, self.ks, self.k_new), (self.v, self.vs, self.v_new)):
            c, s = U.values(codes), scale.double().cpu().numpy()
            added = K.append(c, s, x.double().cpu().numpy(), self.table.cpu().numpy(), self.start, self.off, self.bs, st0)
            want.append((c, s))
        self.run()
        for (c, s), codes, scale in zip(want, (self.k, self.v), (self.ks, self.vs)):
            np.testing.assert_array_equal(scale.double().cpu().numpy(), s)
            np.testing.assert_array_equal(U.values(codes), c)
        assert self.status.cpu().tolist() == [int(a) | b for a, b in zip(st0, added)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,d,H", [(16, 128, 2), (16, 64, 3), (32, 128, 1), (64, 128, 5), (128, 256, 2), (1, 16, 2), (7, 48, 9), (1000, 128, 1)])
def test_append_shapes(bs, d, H, dtype):
    AppendCase([0, 5, 37, 16, 63], [1, 40, 3, 16, 130], H=H, d=d, bs=bs, dtype=dtype).check()


def test_append_single_tokens_and_empty_requests():
    AppendCase([0, 15, 16, 17, 31, 255, 4], [1, 1, 0, 1, 1, 1, 0]).check()


def test_append_many_requests():
    rng = np.random.default_rng(4)
    AppendCase(rng.integers(0, 90, 700).tolist(), rng.integers(0, 4, 700).tolist(), H=1, d=32).check()


def test_append_long_prompt_in_wide_windows():
    # enough tokens that a CTA's window is a whole block
    AppendCase([3, 0, 250], [5000, 777, 9000], H=32, d=128).check()


def test_append_ignores_rows_behind_the_last_sequence():
    c = AppendCase([2, 9], [5, 6], pad=21)
    c.k_new[11:] = float("nan")
    c.check()


def test_append_from_a_fused_projection():
    AppendCase([2, 9, 30], [5, 40, 1], H=3, fused=True).check()
    AppendCase([2, 9, 30], [5, 40, 1], H=3, fused=True, dtype=torch.float32, bs=64).check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_special_values(dtype):
    c = AppendCase([7, 0, 5, 0, 0, 3], [4, 3, 3, 20, 2, 2], dtype=dtype, seed=3)
    c.k_new[0, 0, 5], c.k_new[1, 1, 7], c.v_new[2, 0, 0] = float("inf"), float("-inf"), float("nan")
    c.k_new[4:7] = 0                     # a fresh block of zeros
    c.v_new[7:10] = 1e-38                # far below the smallest scale's subnormals
    c.k_new[7:10, 0] = 3e38              # saturates at the largest scale
    c.v_new[30:32] = float("nan")        # nothing finite
    c.check()


def test_append_keeps_a_scale_that_is_no_power_of_two():
    c = AppendCase([7, 3], [4, 5], seed=5)
    c.ks *= 0.37
    c.vs *= 1e-3                         # grows: the earlier rows are requantised by a rounded ratio
    c.check()


def test_append_twice_is_idempotent():
    c = AppendCase([7, 3], [40, 5], seed=6)
    c.check()
    before = (c.k.view(torch.uint8).clone(), c.ks.clone(), c.v.view(torch.uint8).clone(), c.vs.clone())
    c.run()
    for a, b in zip(before, (c.k.view(torch.uint8), c.ks, c.v.view(torch.uint8), c.vs)):
        assert torch.equal(a, b)


def test_append_data_errors():
    c = AppendCase([4, -3, 5, 2, 60, 8], [20, 4, 3, 40, 30, 4], seed=7, width=4)   # 60 + 30 slots: beyond 4 pages
    c.table[0, 1] = 9999                 # rows of that page only are left out
    c.table[3, 0] = -1
    c.status[2] = 4                      # flagged by an earlier call: not touched
    c.check()
    st = c.status.cpu().tolist()
    assert st[0] == 32 and st[1] == 2 and st[2] == 4 and st[3] == 32 and st[4] == 32 and st[5] == 0


def test_append_inconsistent_offsets():
    c = AppendCase([0, 0, 0], [6, 6, 6], seed=8)
    c.off = np.array([0, 6, 12, 30])     # the last request claims rows past N
    c.check()
    assert c.status.cpu().tolist() == [0, 0, 2]


def test_append_on_another_stream_and_in_a_graph():
    a, b = AppendCase([7, 3, 31], [4, 35, 1], seed=9), AppendCase([7, 3, 31], [4, 35, 1], seed=9)
    a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    start, off = U.ints(b.start), U.ints(b.off.tolist())
    p = B.kv8_append_params(b.k_new, b.v_new, b.k, b.v, b.ks, b.vs, b.table, start, off, b.status)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        B.spec_kv8_append(p, side)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8)) and torch.equal(a.vs, b.vs)


# --------------------------------------------------------------------------------- attention
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 4), (8, 2), (8, 1), (16, 1), (5, 1), (14, 2), (6, 2)])
@pytest.mark.parametrize("T", [1, 5])
def test_attention_head_layouts(Hq, H, T):
    c = U.AttnCase([0, 1, 15, 16, 130, 300], [T] * 6, Hq, H)
    c.run()
    U.check_attention(c)
    assert c.status.cpu().tolist() == [0] * 6


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("sizes", [[1, 1, 1], [3, 1, 7], [40, 17, 64], [129, 5, 256]])
def test_attention_block_sizes(bs, sizes):
    c = U.AttnCase([0, 127, 401], sizes, 4, 2, bs=bs, seed=bs)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("d,bs,Hq,H,dtype", [(64, 16, 4, 2, torch.bfloat16), (128, 16, 4, 2, torch.float32), (256, 16, 4, 1, torch.bfloat16),
                                             (48, 7, 3, 1, torch.float32), (16, 1, 2, 2, torch.float32), (128, 24, 34, 1, torch.bfloat16),
                                             (128, 256, 4, 4, torch.bfloat16)])
def test_attention_other_shapes(d, bs, Hq, H, dtype):
    c = U.AttnCase([0, 33, 500], [1, 6, 20], Hq, H, d=d, bs=bs, dtype=dtype, seed=d)
    c.run()
    U.check_attention(c)


def test_attention_long_prefixes_are_split_and_joined():
    c = U.AttnCase([9001, 3, 4100], [1, 1, 1], 8, 2, seed=11)
    c.run()
    U.check_attention(c)
    c = U.AttnCase([5003, 70], [34, 9], 4, 2, seed=12)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("Hq,H", [(4, 1), (12, 3), (8, 2), (32, 2)])
def test_attention_several_row_tiles(Hq, H):
    """Row tiles in pairs, odd last ones shared out by heads, odd numbers of heads."""
    c = U.AttnCase([700, 3, 129, 0], [70, 200, 9, 33], Hq, H, seed=25)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("Hq,H,T", [(1, 1, 32), (2, 2, 17), (8, 2, 8), (16, 1, 2), (6, 2, 10), (14, 2, 3), (9, 1, 2)])
def test_attention_units_of_17_to_32_rows(Hq, H, T):
    """The rows between the two forms' bounds: prefixes around tiles, split ones, smaller trees, masks."""
    c = U.AttnCase([0, 5, 119, 128, 1500, 300], [T, 1, T, T - 1, T, T], Hq, H, seed=Hq + T)
    c.run()
    U.check_attention(c)
    rng = np.random.default_rng(T)
    bits = [int(rng.integers(0, 1 << T)) if i % 3 else 0 for i in range(2 * T)]
    c = U.AttnCase([0, 121], [T, T], Hq, H, bits=bits, seed=Hq)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("q_scale,spread", [(20.0, 2), (1e-20, 3), (1.0, 60)])
def test_attention_units_of_24_rows_of_unlike_magnitudes(q_scale, spread):
    c = U.AttnCase([900, 77, 2000], [6, 6, 2], 8, 2, q_scale=q_scale, spread=spread, seed=26)
    if spread == 60:
        c.ks.mul_(2.0 ** -50)          # the scores stay finite: only V's scales spread
        c.ks.clamp_(min=2.0 ** -12, max=2.0 ** -8)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("Hq,H", [(32, 1), (40, 2), (71, 1), (128, 1), (130, 1), (192, 3)])
@pytest.mark.parametrize("T", [1, 9])
def test_attention_many_query_heads_of_a_kv_head(Hq, H, T):
    """Row tiles of few tokens, down to one; past 128 heads the CUDA-core kernel."""
    c = U.AttnCase([0, 130, 700], [T, T, 1], Hq, H, seed=Hq)
    c.run()
    U.check_attention(c)


def test_attention_many_requests():
    rng = np.random.default_rng(5)
    c = U.AttnCase(rng.integers(0, 60, 600).tolist(), rng.integers(1, 3, 600).tolist(), 2, 1, seed=13)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("T", [2, 6, 40])
def test_attention_rows_that_see_nothing(T):
    bits = [0] * T + U.chain_bits(T) + [0] * T
    c = U.AttnCase([0, 5, 0], [T] * 3, 4, 2, bits=bits, seed=14)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("T", [6, 40])
def test_attention_arbitrary_masks(T):
    rng = np.random.default_rng(15)
    bits = [int.from_bytes(rng.bytes(8), "little") & ((1 << T) - 1) for _ in range(2 * T)]
    c = U.AttnCase([0, 118], [T, T], 4, 1, bits=bits, T_max=64, seed=15)
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("T", [1, 30])
@pytest.mark.parametrize("q_scale,spread", [(20.0, 2), (1e-3, 20), (1e-20, 3), (1.0, 60)])
def test_attention_magnitudes(T, q_scale, spread):
    """Peaked and flat rows, tiny queries, block scales that differ by many binades."""
    c = U.AttnCase([400, 77], [T, T], 4, 2, q_scale=q_scale, spread=spread, seed=16)
    if spread == 60:
        c.ks.mul_(2.0 ** -50)          # the scores stay finite: only V's scales spread
        c.ks.clamp_(min=2.0 ** -12, max=2.0 ** -8)
    c.run()
    U.check_attention(c)


def test_attention_rows_of_very_different_size():
    c = U.AttnCase([200], [4], 4, 1, seed=17)
    c.q *= torch.tensor([1.0, 1e-6, 1e6, 0.0], device="cuda").to(torch.bfloat16)[None, :, None]
    c.q[:, 2] *= 1e-5
    c.run()
    U.check_attention(c)


@pytest.mark.parametrize("where", ["k", "v", "q", "all keys"])
@pytest.mark.parametrize("Hq,H,T,dtype", [(4, 2, 4, torch.bfloat16), (8, 2, 4, torch.bfloat16), (8, 2, 30, torch.bfloat16),
                                          (16, 2, 60, torch.bfloat16), (6, 2, 6, torch.float32)])
def test_attention_nan_of_one_branch(Hq, H, T, dtype, where):
    """A NaN in a tree node's row reaches the rows that see the node, and no others."""
    rng = np.random.default_rng(T)
    trees = [U.tree_bits(T, rng) for _ in range(3)]
    c = U.AttnCase([3000, 125, 0], [T] * 3, Hq, H, bits=[b for t in trees for b in t], dtype=dtype, seed=T + Hq)
    hit = []
    for r, (P, node) in enumerate(zip(c.prefix, (1, T - 1, T // 2))):
        o = r * T
        hit += [o + i for i in range(T) if (trees[r][i] >> node) & 1]
        page, row = int(c.table_np[r][(P + node) // 16]), (P + node) % 16
        if where == "q":
            hit = hit[:-sum((b >> node) & 1 for b in trees[r])] + [o + node]
            c.q[o + node, :, 77] = float("nan")
        elif where == "all keys" and r < 2:            # a request whose prefix has nothing but NaN scores
            hit = [n for n in hit if n < o] + list(range(o, o + T))
            for s in range(P + T):
                c.k.view(torch.uint8)[int(c.table_np[r][s // 16]), :, s % 16, 3] = 0xFF
        else:
            cache = c.v if where == "v" else c.k
            cache.view(torch.uint8)[page, :, row, 5] = 0x7F
            cache.view(torch.uint8)[page, :, row, 126] = 0xFF
    clean = [n for n in range(c.N) if n not in hit]
    assert hit and (clean or where == "all keys")
    c.run()
    assert c.status.cpu().tolist() == [0] * 3
    o, lse = c.o[hit].float(), c.lse[hit]
    if where == "v":
        assert torch.isnan(o[..., 5]).all() and torch.isnan(o[..., 126]).all() and torch.isfinite(lse).all()
    else:
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    q = c.q.clone()
    c.q = torch.nan_to_num(q, nan=0.0)                 # (the oracle's copy; these rows are not compared)
    if clean:
        U.check_attention(c, rows=clean)


def test_a_pool_of_one_block():
    for dtype in (torch.bfloat16, torch.float32):
        k, v = (torch.full((1, 2, 16, 128), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.full((1, 2), float("nan"), device="cuda") for _ in range(2))
        x = torch.randn((3, 2, 128), device="cuda").to(dtype)
        table, st, start, off = U.ints([0]).view(1, 1), U.ints([0]), U.ints([0]), U.ints([0, 3])
        B.spec_kv8_append(B.kv8_append_params(x, x, k, v, ks, vs, table, start, off, st))
        o, lse = torch.empty_like(x), torch.empty((3, 2), device="cuda")
        p = B.attention_kv8_params(x, k, v, ks, vs, table, start, off, U.mask_words([1, 2, 4], 3), 3, o, lse, st)
        B.spec_tree_attention_kv8(p, torch.empty(max(256, B.spec_attention_kv8_workspace_size(p)), dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        want = v.view(U.E4M3).float()[0, :, :3].transpose(0, 1) * vs[0][None, :, None]
        # (one key a row: its V row, the weight's two pieces and the output's rounding apart)
        assert st.cpu().tolist() == [0] and (o.float() - want).abs().max() <= 2.0 ** -6 * want.abs().max()


def test_attention_refuses_a_workspace_elsewhere():
    c = U.AttnCase([30], [1], 4, 2)
    with pytest.raises(ValueError, match="workspace"):
        B.spec_tree_attention_kv8(c.params(), torch.empty(1 << 24, dtype=torch.uint8))


def test_attention_explicit_scale_and_no_lse():
    c = U.AttnCase([200, 4], [3, 20], 4, 2, seed=18)
    c.run(scale=0.02)
    U.check_attention(c, scale=float(np.float32(0.02)))
    o = c.o.clone()
    c.o.fill_(0)
    c.lse.fill_(5.0)
    c.run(scale=0.02, lse=None)
    assert torch.equal(o, c.o) and (c.lse == 5.0).all()


@pytest.mark.parametrize("T", [1, 3, 20, 60])
def test_attention_leaves_rows_behind_the_last_sequence(T):
    c = U.AttnCase([30, 61], [T, T], 8, 2, pad_rows=9, seed=19)
    c.run()
    U.check_attention(c)
    assert (c.o[c.N:] == 77).all() and (c.lse[c.N:] == 55).all()


@pytest.mark.parametrize("T", [1, 4, 24])
def test_attention_flagged_and_inconsistent_requests(T):
    c = U.AttnCase([30, 61, 200, 9, 40], [T] * 5, 4, 2, seed=20, width=14)
    c.status[1] = 1                     # an earlier call refused its tree
    c.prefix_t[3] = -5
    c.table[2, 3] = 12345               # a page outside the pool
    c.prefix_t[4] = 2000                # slots beyond the table row
    c.run()
    st = c.status.cpu().tolist()
    assert st == [0, 1, 32, 0, 32]
    for r in (1, 3, 4):
        assert (c.o[r * T:(r + 1) * T] == 77).all()
    c.prefix = [30, 0, 0, 0, 0]
    c.table_np = np.maximum(c.table_np, 0)
    U.check_attention(c, rows=slice(0, T))


def test_attention_larger_t_max_than_any_tree():
    for T_max in (64, 256):
        c = U.AttnCase([30, 61], [3, 20], 4, 2, T_max=T_max, seed=21)
        c.run()
        U.check_attention(c)


def test_attention_trees_beyond_t_max_are_left_out():
    c = U.AttnCase([30, 61], [3, 20], 4, 2, seed=22)
    c.T_max = 8
    c.anc = c.anc[:, :1].contiguous()
    c.run()
    assert (c.o[3:] == 77).all() and (c.o[:3] != 77).all()


def test_attention_two_streams_with_a_workspace_each_and_graph_replays():
    a = U.AttnCase([700, 61], [1, 1], 8, 2, seed=23)
    b = U.AttnCase([900, 333], [20, 20], 8, 2, seed=24)
    want = [t.clone() for t in a.run() + b.run()]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    graphs = []
    for c, s in ((a, s1), (b, s2)):
        c.o.zero_()
        c.p = c.params()
        c.ws = torch.empty(max(256, B.spec_attention_kv8_workspace_size(c.p)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for c, s in ((a, s1), (b, s2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            B.spec_tree_attention_kv8(c.p, c.ws, s)
        graphs.append(g)
    for _ in range(5):
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
    torch.cuda.synchronize()
    for t, w in zip((a.o, a.lse, b.o, b.lse), want):
        assert torch.equal(t, w)


# -------------------------------------------------------------------------------- compaction
class CompactCase:
    def __init__(self, prefix, T, n_acc, L=2, H=2, d=128, bs=16, seed=0, paths=None):
        rng = np.random.default_rng(seed)
        Bn = len(prefix)
        need = [-(-(p + T) // bs) for p in prefix]
        nb = sum(need) + 2
        self.table_np = U.table_for(need, nb, rng)
        self.k, self.ks = U.random_cache(L, nb, H, bs, d, rng)
        self.v, self.vs = U.random_cache(L, nb, H, bs, d, rng)
        path = np.full((Bn, T), -1, dtype=np.int32)
        for r in range(Bn):
            if paths is not None:
                path[r, :len(paths[r])] = paths[r]
            elif n_acc[r] >= 0:
                path[r, 0] = 0
                path[r, 1:n_acc[r] + 1] = np.sort(rng.permutation(np.arange(1, T))[:n_acc[r]])
        self.path, self.n_acc, self.prefix, self.bs, self.T = path, n_acc, prefix, bs, T
        self.status = torch.zeros(Bn, dtype=torch.int32, device="cuda")
        self.out = [torch.full((Bn,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
        self.moves = torch.full((Bn, T, 2), -7, dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(self.table_np).cuda()

    def run(self):
        self.held = (U.ints(self.prefix), torch.from_numpy(self.path).cuda(), U.ints(self.n_acc))
        p = B.kv8_compact_params(self.k, self.v, self.ks, self.vs, self.table, self.held[0], self.held[1], self.held[2],
                                 self.status, self.out[0], self.moves, self.out[1], self.T)
        B.spec_kv8_compact(p)
        torch.cuda.synchronize()

    def check(self, status=None):
        st0 = self.status.cpu().tolist()
        status = st0 if status is None else status
        n_ok = [n if s == 0 and n < self.T else -1 for n, s in zip(self.n_acc, status)]
        want = []
        for codes, scale in ((self.k, self.ks), (self.v, self.vs)):
            c, s = U.values(codes), scale.double().cpu().numpy()
            for layer in range(c.shape[0]):
                K.compact(c[layer], s[layer], self.table.cpu().numpy(), self.prefix, self.path, n_ok, self.bs)
            want.append((c, s))
        self.run()
        for (c, s), codes, scale in zip(want, (self.k, self.v), (self.ks, self.vs)):
            np.testing.assert_array_equal(scale.double().cpu().numpy(), s)
            np.testing.assert_array_equal(U.values(codes), c)
        assert self.status.cpu().tolist() == status
        lens = [p + n + 1 if n >= 0 else p for p, n in zip(self.prefix, n_ok)]
        assert self.out[0].cpu().tolist() == lens
        assert self.out[1].cpu().tolist() == [-(-n // self.bs) for n in lens]
        m = self.moves.cpu().numpy()
        for r, (p, n) in enumerate(zip(self.prefix, n_ok)):
            for d in range(self.T):
                assert m[r, d].tolist() == ([p + self.path[r, d], p + d] if d <= n else [-1, -1])


@pytest.mark.parametrize("bs,d,H", [(16, 128, 2), (32, 128, 5), (64, 64, 1), (128, 256, 2), (4, 16, 3), (1, 48, 2), (300, 128, 1)])
def test_compact_shapes(bs, d, H):
    CompactCase([0, 15, 16, 37, 200], 40, [0, 7, 3, 39, 12], H=H, d=d, bs=bs).check()


def test_compact_long_paths():
    CompactCase([3, 130], 256, [255, 200], L=1, H=1, bs=64, seed=2).check()


def test_compact_partly_identical_paths_and_repeats():
    CompactCase([5, 12, 30], 20, [3, 5, 4], paths=[[0, 1, 2, 3], [0, 1, 2, 9, 10, 17], [0, 6, 6, 6, 8]], seed=3).check()


def test_compact_scales_that_are_no_powers_of_two():
    c = CompactCase([5, 12], 20, [3, 5], seed=4)
    c.ks *= 0.37
    c.vs *= torch.rand_like(c.vs) + 0.5
    c.check()


def test_compact_rollback_and_data_errors():
    c = CompactCase([5, 12, 30, 8, 16, 7], 20, [3, -1, 4, 2, 3, 25], seed=5)
    c.status[0] = 4
    c.path[3, 1] = 0                      # not above its step
    c.table[4] = -1
    c.check(status=[4, 0, 0, 1, 32, 0])


# -------------------------------------------------------------------------------------- fork
class ForkCase:
    def __init__(self, lens, src, dst, dtype="e4m3", L=2, H=2, d=128, bs=16, seed=0, fresh=None):
        rng = np.random.default_rng(seed)
        need = [-(-n // bs) for n in lens]
        F = len(src)
        nb = sum(need) + F + 2
        t = U.table_for(need, sum(need) or 1, rng, width=max(need) + 1)
        self.table = torch.from_numpy(t).cuda()
        self.fresh = [sum(need) + i for i in rng.permutation(F)] if fresh is None else fresh
        self.ks = self.vs = None
        if dtype == "e4m3":
            self.k, self.ks = U.random_cache(L, nb, H, bs, d, rng)
            self.v, self.vs = U.random_cache(L, nb, H, bs, d, rng)
        else:
            td = torch.bfloat16 if dtype == "bf16" else torch.float32
            self.k, self.v = (torch.from_numpy(rng.normal(size=(L, nb, H, bs, d))).to(td).cuda() for _ in range(2))
        self.lens, self.src, self.dst, self.bs = lens, src, dst, bs
        self.kv_len = U.ints(lens)
        self.status = torch.full((F,), -7, dtype=torch.int32, device="cuda")

    def bits(self):
        es = self.k.element_size()
        as_int = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[es]
        return [t.view(as_int) for t in (self.k, self.v)] + ([self.ks, self.vs] if self.ks is not None else [])

    def check(self, status=None):
        status = status or [0] * len(self.src)
        want = [t.clone() for t in self.bits()]
        table, kv = self.table.clone(), list(self.lens)
        for f, (a, c) in enumerate(zip(self.src, self.dst)):
            if status[f]:
                continue
            full, rem = self.lens[a] // self.bs, self.lens[a] % self.bs
            table[c, :full] = self.table[a, :full]
            kv[c] = self.lens[a]
            if rem:
                pb, nb = int(self.table[a, full]), self.fresh[f]
                table[c, full] = nb
                for t in want[:2]:
                    t[:, nb, :, :rem] = t[:, pb, :, :rem]
                for t in want[2:]:
                    t[:, nb] = t[:, pb]
        held = (U.ints(self.src), U.ints(self.dst), U.ints(self.fresh))
        B.spec_kv_fork(B.kv_fork_params(self.k, self.v, self.table, self.kv_len, *held, self.status, self.ks, self.vs))
        torch.cuda.synchronize()
        assert self.status.cpu().tolist() == status
        assert self.kv_len.cpu().tolist() == kv and torch.equal(self.table, table)
        for t, w in zip(self.bits(), want):
            assert torch.equal(t, w)


@pytest.mark.parametrize("dtype", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("bs,d,H", [(16, 128, 2), (64, 128, 3), (7, 16, 1), (16, 48, 40)])
def test_fork_shapes(dtype, bs, d, H):
    ForkCase([0, 1, 15, 16, 100, 3, 3, 3, 3, 3, 3], [0, 1, 2, 3, 4, 4], [5, 6, 7, 8, 9, 10], dtype, H=H, d=d, bs=bs).check()


def test_fork_many():
    n = 300
    ForkCase([100 + i for i in range(4)] + [0] * n, [i % 4 for i in range(n)], [4 + i for i in range(n)], L=1, H=1, d=16).check()


def test_fork_refuses_what_would_depend_on_order():
    # 0: fine; 1: child twice; 2: child twice; 3: child is a parent of another; 4: bad ids; 5: itself
    ForkCase([20, 20, 20, 20, 20, 20, 20], [0, 0, 0, 1, 9, 6], [2, 3, 3, 0, 4, 6]).check([0, 1, 1, 1, 1, 1])


def test_fork_refuses_bad_pages_and_lengths():
    c = ForkCase([20, 20, 20, 20, 32, 20, 20, 20, 20, 20, 20], [0, 1, 2, 3, 4], [5, 6, 7, 8, 9], seed=3)
    c.fresh[0] = 9999
    c.fresh[1] = int(c.table[1, 0])
    c.table[2, 0] = -1
    c.fresh[4] = -1                       # whole pages only: no fresh page is read
    c.check([32, 32, 32, 0, 0])
    c = ForkCase([20, 20, 20, 20, 16], [0, 1, 4], [2, 3, 0], seed=4, fresh=[6, 6, 6])
    c.dst = [2, 3, 0]
    c.src = [1, 1, 4]
    c.check([1, 1, 0])                    # one fresh page for two copies; the third copies nothing
    c = ForkCase([20, 20, 20], [0], [1], seed=5)
    c.lens[0] = -4
    c.kv_len[0] = -4
    c.check([2])


# ------------------------------------------------------------------------------ far addresses
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slots_at_the_end_of_32_bits_are_refused(dtype):
    """A table row of 2^27 - 1 pages of 16: the slots' numbers fit, a tile past them does not."""
    H, d, P, T = 1, 128, 2 ** 31 - 25, 5
    table = torch.zeros((1, 2 ** 27 - 1), dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((1, 4, H, 16, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((1, 4, H), device="cuda") for _ in range(2))
    x = torch.ones((T, H, d), device="cuda").to(dtype)
    pre, off = U.ints([P]), U.ints([0, T])
    st = [U.ints([0]) for _ in range(2)]
    o, lse = torch.full_like(x, 77.0), torch.full((T, H), 55.0, device="cuda")
    p = B.attention_kv8_params(x, k[0], v[0], ks[0], vs[0], table, pre, off, U.mask_words(U.chain_bits(T), T), T, o, lse, st[0])
    B.spec_tree_attention_kv8(p, torch.empty(max(256, B.spec_attention_kv8_workspace_size(p)), dtype=torch.uint8, device="cuda"))
    outs = [U.ints([0]), torch.zeros((1, 3, 2), dtype=torch.int32, device="cuda"), U.ints([0])]
    path = torch.tensor([[0, 2, 4]], dtype=torch.int32, device="cuda")
    B.spec_kv8_compact(B.kv8_compact_params(k, v, ks, vs, table, pre, path, U.ints([2]), st[1], *outs, 3))
    torch.cuda.synchronize()
    assert [s.item() for s in st] == [32, 1] and outs[0].item() == P
    assert (o == 77).all() and (lse == 55).all() and (k == 0).all() and (v == 0).all() and (ks == 1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_beyond_four_gigabytes(dtype):
    """The same calls on a small pool and on one whose pages lie past 2^32 bytes: bit for bit alike."""
    H, Hq, bs, d, L, far = 8, 16, 16, 128, 2, 2 ** 32 // (8 * 16 * 128)
    start, n = [0, 37, 200], [50, 6, 1]
    off = np.concatenate([[0], np.cumsum(n)]).tolist()
    g = torch.Generator(device="cuda").manual_seed(50)
    kn, vn = (torch.randn((off[-1], H, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((off[-1], Hq, d), generator=g, device="cuda").to(dtype)
    rng = np.random.default_rng(51)
    ids = U.table_for([5, 5, 15], 40, rng, 16)
    seeds = [U.random_cache(1, 40, H, bs, d, rng, junk=False) for _ in range(2)]
    results = []
    for shift in (0, far):
        nb = 40 + shift
        (k, ks), (v, vs) = [(torch.zeros((L, nb, H, bs, d), dtype=torch.uint8, device="cuda"), torch.zeros((L, nb, H), device="cuda"))
                            for _ in range(2)]
        for (c, s), (c0, s0) in zip(((k, ks), (v, vs)), seeds):
            c[1, shift:] = c0[0].view(torch.uint8)
            s[1, shift:] = s0[0]
        k, v = k.view(U.E4M3), v.view(U.E4M3)
        table = torch.from_numpy(np.where(ids >= 0, ids + shift, ids).astype(np.int32)).cuda()
        st = torch.zeros(3, dtype=torch.int32, device="cuda")
        held = (U.ints(start), U.ints(off))
        B.spec_kv8_append(B.kv8_append_params(kn, vn, k[1], v[1], ks[1], vs[1], table, *held, st))
        o, lse = torch.zeros_like(q), torch.zeros((off[-1], Hq), device="cuda")
        bits = [b for t in n for b in U.chain_bits(t)]
        p = B.attention_kv8_params(q=q, k_cache=k[1], v_cache=v[1], k_scale=ks[1], v_scale=vs[1], block_table=table,
                                   prefix_len=held[0], node_offset=held[1], anc_mask=U.mask_words(bits, 50), T_max=50, o=o, lse=lse,
                                   req_status=st)
        B.spec_tree_attention_kv8(p, torch.empty(max(256, B.spec_attention_kv8_workspace_size(p)), dtype=torch.uint8, device="cuda"))
        path = torch.tensor([[0, 5, 49], [0, 3, 5], [0, 0, 0]], dtype=torch.int32, device="cuda")
        outs = [U.ints([0] * 3), torch.zeros((3, 3, 2), dtype=torch.int32, device="cuda"), U.ints([0] * 3)]
        B.spec_kv8_compact(B.kv8_compact_params(k, v, ks, vs, table, held[0], path, U.ints([2, 2, 0]), st, *outs, 3))
        lens, fs = outs[0].clone(), U.ints([0])
        wide = torch.cat([table, torch.full_like(table[:1], -1)])
        lens = torch.cat([lens, U.ints([0])])
        fresh = int(np.setdiff1d(np.arange(40), ids)[0])
        B.spec_kv_fork(B.kv_fork_params(k, v, wide, lens, U.ints([1]), U.ints([3]), U.ints([fresh + shift]), fs, ks, vs))
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [0] * 3 and fs.cpu().tolist() == [0] and lens.cpu().tolist() == [3, 40, 201, 40]
        back = [t[:, shift:].cpu() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
        results.append([o.cpu(), lse.cpu(), outs[1].cpu(), wide.cpu() - shift * (wide.cpu() >= 0).int()] + back)
        del k, v, ks, vs, p
        torch.cuda.empty_cache()
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------------- together
def test_a_decoding_loop_over_the_cache():
    """Prompt, forked samples, single tokens: append -> fork -> append -> attention, each step against
    the oracle run on the same rows from the start."""
    H, Hq, bs, d = 2, 8, 16, 128
    rng = np.random.default_rng(31)
    g = torch.Generator(device="cuda").manual_seed(31)
    nb, prompt, forks, steps = 40, 37, 3, 20
    Bn = 1 + forks
    k, ks = torch.zeros((1, nb, H, bs, d), device="cuda").to(E4M3), torch.zeros((1, nb, H), device="cuda")
    v, vs = torch.zeros_like(k), torch.zeros_like(ks)
    ids = rng.permutation(nb)
    table_np = np.full((Bn, 5), -1, dtype=np.int32)
    table_np[0] = ids[:5]
    for r in range(1, Bn):
        table_np[r, 3:] = ids[5 + 3 * r:7 + 3 * r]
    table, status = torch.from_numpy(table_np).cuda(), torch.zeros(Bn, dtype=torch.int32, device="cuda")
    rows = lambda n: torch.randn((n, H, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ok, oks, ov, ovs = U.values(k)[0], ks[0].double().cpu().numpy(), U.values(v)[0], vs[0].double().cpu().numpy()

    def append(kn, vn, start, off):
        args = (U.ints(start), U.ints(off))
        B.spec_kv8_append(B.kv8_append_params(kn, vn, k[0], v[0], ks[0], vs[0], table, *args, status))
        K.append(ok, oks, kn.double().cpu().numpy(), table.cpu().numpy(), start, off, bs)
        K.append(ov, ovs, vn.double().cpu().numpy(), table.cpu().numpy(), start, off, bs)
        torch.cuda.synchronize()

    append(rows(prompt), rows(prompt), [0] * Bn, [0] + [prompt] * Bn)
    kv_len, fs = U.ints([prompt] + [0] * forks), torch.zeros(forks, dtype=torch.int32, device="cuda")
    fresh = [int(ids[5 + 3 * r + 2]) for r in range(1, Bn)]
    held = (U.ints([0] * forks), U.ints(list(range(1, Bn))), U.ints(fresh))
    B.spec_kv_fork(B.kv_fork_params(k, v, table, kv_len, *held, fs, ks, vs))
    torch.cuda.synchronize()
    assert fs.cpu().tolist() == [0] * forks and kv_len.cpu().tolist() == [prompt] * Bn
    last = int(table_np[0, prompt // bs])
    for nbk in fresh:
        for arr in (ok, ov):
            arr[nbk, :, :prompt % bs] = arr[last, :, :prompt % bs]
        oks[nbk], ovs[nbk] = oks[last], ovs[last]
    for step in range(steps):
        P = prompt + step
        append(rows(Bn), rows(Bn), [P] * Bn, list(range(Bn + 1)))
        np.testing.assert_array_equal(U.values(k)[0], ok)
        np.testing.assert_array_equal(vs[0].double().cpu().numpy(), ovs)
        if step % 7 == 0:
            c = U.AttnCase([P] * Bn, [1] * Bn, Hq, H, seed=step, poison=False)
            c.k, c.ks, c.v, c.vs, c.table, c.table_np = k[0], ks[0], v[0], vs[0], table, table.cpu().numpy()
            c.run()
            U.check_attention(c)
    assert status.cpu().tolist() == [0] * Bn


def _round_case(cid, layers, seed=41):
    from speculative_decoding_draft_tree_gb300 import workloads as W
    from speculative_decoding_draft_tree_gb300.api import VerifyStep
    w = W.make_config(cid, scale="small", device="cuda", num_layers=layers)
    rng = np.random.default_rng(seed)
    nb, H, bs, d = w.k_cache.shape[1:]
    k, ks = U.random_cache(layers, nb, H, bs, d, rng, junk=False)
    v, vs = U.random_cache(layers, nb, H, bs, d, rng, junk=False)
    k_new, v_new = W.new_tree_kv(w)
    step = VerifyStep(w)
    step.enable_kv8(k, v, ks, vs, k_new, v_new)
    return w, step, (k, v, ks, vs, k_new, v_new)


@pytest.mark.parametrize("cid", [1, 2, 3, 4, 5])
def test_a_verification_round_over_the_cache(cid):
    """VerifyStep.run over an 8-bit cache: append, attention, verification and compaction against
    the oracles run one after the other."""
    import parity_util as PU
    w, step, (k, v, ks, vs, k_new, v_new) = _round_case(cid, 2)
    snap = PU.snapshot(w)
    no, prefix, table = snap["node_offset"], snap["prefix_len"], snap["block_table"]
    cache = [[U.values(c[layer]), s[layer].double().cpu().numpy()] for c, s in ((k, ks), (v, vs)) for layer in range(2)]
    for (c, s), x in ((cache[0], k_new), (cache[2], v_new)):
        K.append(c, s, x.double().cpu().numpy(), table, prefix, no, w.bs)
    step.run()
    torch.cuda.synchronize()
    PU.check_tree(w, step, snap)
    PU.check_verify(w, step, PU.oracle_verify(w, snap))
    c = U.AttnCase.__new__(U.AttnCase)
    c.N, c.T_max, c.bs, c.prefix, c.off_np, c.table_np = w.N, w.T_max, w.bs, prefix, no, table
    c.q, c.o, c.lse = w.q, step.o, step.lse
    words = step.anc_mask.cpu().numpy().view(np.uint32)
    c.bits = [sum(int(x) << (32 * j) for j, x in enumerate(row)) for row in words]
    # attention ran before the compaction: the oracle takes the appended cache
    c.oracle = lambda scale=None: K.tree_attention(
        w.q.double().cpu().numpy(), cache[0][0], cache[0][1], cache[2][0], cache[2][1], table, prefix, no,
        [[(b >> j) & 1 for j in range(w.T_max)] for b in c.bits], w.bs, scale)
    c.ks = ks[0]
    U.check_attention(c)
    path, n_acc = step.path.cpu().numpy(), step.n_acc.cpu().numpy()
    for (codes, scale), (gc, gs) in zip(cache, [(t[layer], u[layer]) for t, u in ((k, ks), (v, vs)) for layer in range(2)]):
        K.compact(codes, scale, table, prefix, path, n_acc, w.bs)
        np.testing.assert_array_equal(U.values(gc), codes)
        np.testing.assert_array_equal(gs.double().cpu().numpy(), scale)
    assert step.new_kv_len.cpu().tolist() == [int(p) + int(n) + 1 for p, n in zip(prefix, n_acc)]


def test_rounds_over_the_cache_from_a_graph_and_a_pipeline():
    """The same round captured as a graph, and submitted through RoundPipeline, gives run()'s bits."""
    from speculative_decoding_draft_tree_gb300.api import RoundPipeline
    names = ("o", "lse", "out_tokens", "out_len", "path", "n_acc", "new_kv_len", "slot_map")
    w, step, cache = _round_case(4, 1)
    before = [t.clone() for t in cache[:4]]
    step.run()
    torch.cuda.synchronize()
    want = [getattr(step, n).clone() for n in names] + [t.clone() for t in cache[:4]]

    def back():
        for t, b in zip(cache[:4], before):
            t.copy_(b)
    back()
    g = step.capture_graph()
    g.replay()
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    for t, x in zip([getattr(step, n) for n in names] + list(cache[:4]), want):
        assert same(t, x)
    back()
    pipe = RoundPipeline(step)
    i = pipe.submit(pipe.pinned_host_inputs())
    pipe.finish()
    torch.cuda.synchronize()
    out = pipe.host_outputs(i)
    assert torch.equal(out["out_tokens"], want[names.index("out_tokens")].cpu())
    assert torch.equal(out["new_kv_len"], want[names.index("new_kv_len")].cpu())
    for t, x in zip(cache[:4], want[len(names):]):
        assert same(t, x)


def test_enable_kv8_and_enable_rope_exclude_each_other():
    w, step, (k, v, ks, vs, k_new, v_new) = _round_case(2, 1)
    with pytest.raises(ValueError, match="rotated"):
        step.enable_rope(w.q.clone(), k_new, v_new)
    from speculative_decoding_draft_tree_gb300.api import VerifyStep
    other = VerifyStep(w)
    other.enable_rope(w.q.clone(), k_new, v_new)
    with pytest.raises(ValueError, match="enable_rope"):
        other.enable_kv8(k, v, ks, vs, k_new, v_new)


# ------------------------------------------------------------------ refusals of the binding
def test_parameters_hold_their_tensors_and_their_device():
    c = U.AttnCase([20, 3], [2, 4], 4, 2)
    want = c.run()[0].clone()
    p = c.params(q=c.q.clone(), block_table=c.table.clone(), prefix_len=c.prefix_t.clone(), node_offset=c.off.clone())
    junk = [torch.full((1 << 12,), 2 ** 30, dtype=torch.int32, device="cuda") for _ in range(64)]   # takes freed memory
    c.o.zero_()
    B.spec_tree_attention_kv8(p, torch.empty(B.spec_attention_kv8_workspace_size(p), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(c.o, want) and len(junk) == 64
    p._device = 7                         # as if the tensors were on another device than the current one
    with pytest.raises(ValueError, match="current device"):
        B.spec_tree_attention_kv8(p, None)


def test_binding_refuses_wrong_shapes_and_types():
    c = U.AttnCase([20, 3], [2, 4], 4, 2)
    bad = [dict(q=c.q.double()), dict(o=c.o[:1]), dict(lse=c.lse[:, :1]), dict(anc_mask=c.anc[:1]), dict(T_max=64),
           dict(k_scale=c.ks[:1]), dict(v_cache=c.v.float()), dict(k_cache=c.k[:, :, :8].contiguous()),
           dict(prefix_len=c.prefix_t[:1]), dict(node_offset=c.off[:1]), dict(req_status=c.status.long()),
           dict(block_table=c.table.cpu()), dict(q=c.q[:, ::2])]
    for kw in bad:
        with pytest.raises(ValueError):
            c.params(**kw)
    p = c.params()
    with pytest.raises(B.SpecError, match="INVALID_ARG"):          # no workspace
        B.spec_tree_attention_kv8(p, None)
    with pytest.raises(B.SpecError, match="INVALID_ARG"):          # a small one
        B.spec_tree_attention_kv8(p, torch.empty(256, dtype=torch.uint8, device="cuda"))
    a = AppendCase([2], [5])
    with pytest.raises(ValueError, match="contiguous"):
        B.kv8_append_params(a.k_new.transpose(1, 2).contiguous().transpose(1, 2), a.v_new, a.k, a.v, a.ks, a.vs, a.table,
                            U.ints([2]), U.ints([0, 5]), a.status)
    with pytest.raises(ValueError, match="v_new"):
        B.kv8_append_params(a.k_new, a.v_new.float(), a.k, a.v, a.ks, a.vs, a.table, U.ints([2]), U.ints([0, 5]), a.status)
