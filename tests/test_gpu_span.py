"""GPU parity of windowed and shared-prefix attention with the fp64 oracle; bars in span_util.check."""
import numpy as np
import pytest
import torch

import kv8_util as U
import span_util as S
from oracle import span
from speculative_decoding_draft_tree_gb300 import binding as B

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------------------------------ window
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (100, 0), (128, 4), (129, 130), (300, 17), (513, 64), (5000, 0), (1, 5000)])
@pytest.mark.parametrize("T", [1, 6])
def test_window_decoding_and_chains(T, window, sinks):
    c = S.Case([0, 1, 127, 128, 129, 700, 1031], [T] * 7, Hq=8, H=2, window=window, sinks=sinks, seed=window + sinks)
    c.run()
    S.check(c)


@pytest.mark.parametrize("bs,d,G,H,dtype", [(16, 128, 1, 3, BF16), (32, 128, 5, 2, BF16), (64, 128, 7, 1, BF16), (128, 128, 16, 1, BF16),
                                            (16, 128, 128, 1, BF16), (16, 128, 129, 1, BF16), (7, 128, 2, 2, BF16), (16, 64, 4, 2, BF16),
                                            (16, 256, 2, 1, BF16), (1, 40, 3, 2, BF16), (16, 128, 4, 2, F32), (32, 64, 1, 4, F32),
                                            (5, 256, 2, 1, F32), (16, 12, 2, 2, F32)])
def test_window_shapes(bs, d, G, H, dtype):
    c = S.Case([0, 40, 333], [3, 1, 20], Hq=G * H, H=H, d=d, bs=bs, dtype=dtype, window=150, sinks=6, seed=bs + d)
    c.run()
    S.check(c)


@pytest.mark.parametrize("T", [17, 64, 100, 256])
@pytest.mark.parametrize("window,sinks", [(2, 0), (4, 3), (60, 10), (400, 4)])
def test_window_over_trees(T, window, sinks):
    """Depths of these trees pass the smaller windows; sinks that reach into the tree (prefix 1)."""
    c = S.Case([300, 1], [T, max(1, T // 2)], Hq=8, H=2, window=window, sinks=sinks, seed=T + window)
    c.run()
    S.check(c)


def test_window_over_a_deep_chain_in_a_wide_mask():
    c = S.Case([100, 3], [200, 90], Hq=4, H=1, window=33, sinks=5, bits=U.chain_bits(200) + U.chain_bits(90), seed=3)
    c.run()
    S.check(c)


def test_window_splits_long_caches():
    """Few heads and long windows: units are cut, and their pieces merged."""
    c = S.Case([9000, 4000, 20], [1, 1, 1], Hq=8, H=1, window=7000, sinks=300, seed=5)
    c.run()
    S.check(c)
    c = S.Case([5000, 2500], [130, 60], Hq=4, H=1, window=4000, sinks=4, seed=6)
    c.run()
    S.check(c)


def test_window_equals_tree_attention_when_it_is_wide():
    c = S.Case([500, 77, 0], [46, 1, 9], Hq=8, H=2, window=1000, seed=7)
    c.run()
    o, lse = torch.empty_like(c.o), torch.empty_like(c.lse)
    k, v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    p = B.attention_params(c.q, k, v, c.table, c.prefix_t, c.off, c.anc, c.T_max, o, lse, c.status)
    B.spec_tree_attention(p, torch.empty(B.spec_attention_workspace_size(p), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    norm = o.double().norm().item()     # each within 0.0032 of the exact values
    assert (o.double() - c.o.double()).norm().item() <= 6.4e-3 * norm
    assert (lse - c.lse).abs().max().item() < 2e-4


# ------------------------------------------------------------------------------------ shared
@pytest.mark.parametrize("shared", [0, 1, 15, 16, 127, 128, 129, 500])
@pytest.mark.parametrize("T", [1, 5])
def test_shared_decoding_and_chains(T, shared):
    c = S.Case([shared, shared + 1, shared + 130, shared + 17, shared + 40, shared], [T] * 6, Hq=8, H=2, groups=[(0, 3, shared), (3, 4, shared), (4, 6, shared)], seed=shared)
    c.run()
    S.check(c)


@pytest.mark.parametrize("bs,d,G,H,dtype", [(16, 128, 1, 3, BF16), (32, 128, 5, 2, BF16), (64, 128, 7, 1, BF16), (128, 128, 16, 1, BF16),
                                            (16, 128, 128, 1, BF16), (16, 128, 129, 1, BF16), (7, 128, 2, 2, BF16), (16, 64, 4, 2, BF16),
                                            (16, 256, 2, 1, BF16), (1, 40, 3, 2, BF16), (16, 128, 4, 2, F32), (32, 64, 1, 4, F32),
                                            (5, 256, 2, 1, F32), (16, 12, 2, 2, F32)])
def test_shared_shapes(bs, d, G, H, dtype):
    c = S.Case([90, 133, 90, 200], [3, 1, 20, 2], Hq=G * H, H=H, d=d, bs=bs, dtype=dtype, groups=[(0, 3, 90), (3, 4, 11)], seed=bs + d)
    c.run()
    S.check(c)


@pytest.mark.parametrize("members,G", [(33, 4), (65, 4), (70, 8), (40, 5), (3, 128)])
def test_shared_row_tiles(members, G):
    """One row tile, two, three and more of a group's rows; tiles that end between requests."""
    rng = np.random.default_rng(members)
    own = rng.integers(0, 60, members)
    c = S.Case([(300 + int(n)) for n in own], [1 + int(n) % 3 for n in own], Hq=G, H=1, groups=[(0, members, 300)], seed=members)
    c.run()
    S.check(c)


def test_shared_trees_and_groups_of_many_sizes():
    sizes = [46, 1, 100, 17, 256, 3, 30, 60]
    prefix = [700, 650, 1000, 400, 401, 90, 90, 90]
    c = S.Case(prefix, sizes, Hq=8, H=2, groups=[(0, 3, 650), (3, 5, 399), (5, 6, 0), (6, 8, 90)], seed=11)
    c.run()
    S.check(c)


def _few_rows_each(kind, H, T):
    """More (request, head) units of at most 32 rows than two per SM: neighbouring heads share theirs; 3 heads
    leave one alone.  A group of 65 members has 260 rows and more: two full tiles and a small one."""
    n = max(2 * torch.cuda.get_device_properties(0).multi_processor_count // H + 1, 80)
    rng = np.random.default_rng(H * 10 + T)
    prefix = [40 + int(x) for x in rng.integers(0, 300, n)]
    if kind == "window":
        return S.Case(prefix, [T] * n, Hq=4 * H, H=H, window=100, sinks=3, seed=H)
    return S.Case(prefix, [T] * n, Hq=4 * H, H=H, groups=[(0, 8, 40), (8, 73, 33), (73, 74, 17), (74, n, 0)], seed=H)


@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("H,T", [(3, 5), (8, 8), (4, 1), (3, 1)])
def test_many_units_of_few_rows(kind, H, T):
    c = _few_rows_each(kind, H, T)
    c.run()
    S.check(c)


@pytest.mark.parametrize("kind", ["window", "shared"])
def test_a_bad_value_stays_under_its_head(kind):
    """V's infinity in one head's slot does not reach the head that shares the unit, nor other requests."""
    c = _few_rows_each(kind, 3, 5)
    c.run()
    o, lse = c.o.clone(), c.lse.clone()
    r, h = 9, 1
    slot = c.prefix[r] + 1                      # the second node's: it and its descendants see it
    c.v[c.table_np[r, slot // c.bs], h, slot % c.bs, 7] = float("inf")
    c.run()
    hit = torch.zeros(c.o.shape[:2], dtype=torch.bool, device="cuda")
    a = c.off_np[r]
    for i in range(c.sizes[r]):
        hit[a + i, 4 * h:4 * h + 4] = bool((c.bits[a + i] >> 1) & 1)
    assert (~torch.isfinite(c.o[hit][:, 7])).all()
    assert torch.equal(c.o[~hit].view(torch.int16), o[~hit].view(torch.int16)) and torch.equal(c.lse[~hit], lse[~hit])


def test_shared_splits_a_long_prefix():
    c = S.Case([12000, 12100, 12010], [1, 1, 1], Hq=4, H=1, groups=[(0, 3, 12000)], seed=12)
    c.run()
    S.check(c)


def test_shared_reads_the_common_slots_by_the_first_row_only():
    c = S.Case([200, 200, 200], [1, 1, 1], Hq=4, H=2, groups=[(0, 3, 200)], seed=13)
    assert (c.table_np[1:, :12] == -1).all()       # the members' own entries of the shared pages are not read
    c.run()
    S.check(c)
    assert c.status.tolist() == [0, 0, 0]


# ------------------------------------------------------------------------------------ both
def _kinds():
    return [dict(window=90, sinks=3), dict(groups=[(0, 2, 60), (2, 3, 40)])]


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_nothing(kind, dtype):
    """Empty mask rows: with a prefix they see it (or what a window leaves of it), without one nothing."""
    bits = [0, 2, 0] + [0] * 3 + [1, 0, 4]
    kw = dict(kind) if "window" in kind else dict(groups=[(0, 2, 0), (2, 3, 40)])
    c = S.Case([0, 0, 60], [3, 3, 3], Hq=4, H=2, dtype=dtype, bits=bits, seed=20, **kw)
    c.run()
    S.check(c)


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_only_named_rows_are_written(kind, dtype):
    """Rows behind the last sequence, rows of a request that an earlier call flagged."""
    c = S.Case([60, 80, 75], [2, 3, 2], Hq=4, H=2, dtype=dtype, pad_rows=5, seed=21, **kind)
    c.status[1] = 4
    c.run()
    S.check(c, rows=[0, 1, 5, 6])
    assert (c.o[2:5] == 77).all() and (c.lse[2:5] == 55).all() and (c.o[7:] == 77).all() and (c.lse[7:] == 55).all()
    assert c.status.tolist() == [0, 4, 0]


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lse_may_be_missing_and_scale_given(kind, dtype):
    c = S.Case([60, 80, 75], [2, 20, 2], Hq=4, H=2, dtype=dtype, seed=22, **kind)
    c.run(scale=0.21)
    S.check(c, scale=0.21)
    o = c.o.clone()
    c.o.fill_(5)
    c.run(scale=0.21, lse=None)
    assert torch.equal(c.o, o)


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sharp_scores(kind, dtype):
    """One key far above the others, references that move late, weights that underflow."""
    c = S.Case([260, 280, 275], [2, 20, 1], Hq=4, H=2, dtype=dtype, q_scale=12.0, seed=23, **kind)
    c.run()
    S.check(c)


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [20, 4])
def test_nan_and_infinity_reach_the_rows_that_see_them(kind, dtype, T):
    """In q, in a tree node's K or V, and at a prefix slot that a window hides from some rows."""
    c = S.Case([260, 280, 275], [T, T, T], Hq=4, H=2, dtype=dtype, seed=24, **kind)
    slots = [280 + 1, 275 - 86]                        # node 1 of request 1; a prefix slot of request 2
    where = []
    for r, s, t, val in ((1, slots[0], c.v, float("nan")), (2, slots[1], c.v, float("inf")), (2, 275 + 2, c.k, float("nan"))):
        first, ln = r, 0
        for a, b, n in c.groups or []:
            if a <= r < b:
                first, ln = a, n
        page = int(c.table_np[first if s < ln else r, s // c.bs])
        t[page, 1, s % c.bs, 5] = val
        where.append((r, s))
    c.q[2, 0, 7] = float("nan")                         # node 2 of request 0, head 0
    c.run()
    hit = np.zeros((c.N, 4), dtype=bool)
    hit[2, 0] = True
    for r, s in where:
        for i in range(T):
            n = c.off_np[r] + i
            if s in span.visible(c.bits[n], c.prefix[r], T, c.window, c.sinks):
                hit[n, 2:] = True                       # KV head 1
    o = c.o.double().cpu().numpy()
    assert hit.any() and not hit.all()
    assert (~np.isfinite(o).all(axis=2) == hit).all()
    # the others are what they are without the bad elements (masked there all the same)
    clean = c.o.clone()
    for t in (c.k, c.v):
        t.masked_fill_(t.isinf(), 0.0)
    c.q[2, 0, 7] = 0.0
    c.k.nan_to_num_()
    c.v.nan_to_num_()
    c.run()
    same = torch.from_numpy(~hit).cuda()
    assert torch.equal(clean[same], c.o[same])
    S.check(c)


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
def test_data_errors(kind):
    B_, N = 6, 12
    kw = dict(window=90, sinks=3) if "window" in kind else dict(groups=[(0, 1, 0), (1, 2, 0), (2, 4, 60), (4, 6, 60)])
    c = S.Case([60, 200, 100, 120, 130, 61], [2] * B_, Hq=4, H=2, seed=25, **kw)
    c.prefix_t[0] = -1                                   # BAD_SIZE
    c.table[1, 200 // 16] = 10 ** 6                      # the tree's page: BAD_BLOCK
    c.prefix_t[5] = 10 ** 6                              # beyond the table row: BAD_BLOCK
    c.run()
    assert c.status.tolist() == [2, 32, 0, 0, 0, 32]
    S.check(c, rows=list(range(4, 10)))
    assert (c.o[:2] == 77).all() and (c.o[10:] == 77).all()


def test_window_does_not_look_at_pages_out_of_sight():
    c = S.Case([1000, 600], [3, 1], Hq=4, H=2, window=100, sinks=20, seed=26)
    hidden = c.table_np < 0
    assert hidden[0, 2:55].all()
    for junk in (-5, 10 ** 8):
        c.table[torch.from_numpy(hidden).cuda()] = junk
        c.run()
        S.check(c)
        assert c.status.tolist() == [0, 0]


def test_shared_data_errors():
    """A shared length beyond a member's prefix, a negative one, groups that leave a request out or overlap, a
    bad shared page."""
    mk = lambda: S.Case([60, 40, 90, 100, 80], [1, 2, 1, 1, 2], Hq=4, H=2, groups=[(0, 2, 30), (2, 4, 50), (4, 5, 10)], seed=27)  # noqa: E731
    c = mk()
    c.shared[0], c.shared[2] = 50, -1
    c.run()
    assert c.status.tolist() == [0, 2, 0, 0, 2]
    assert (c.o[1:3] == 77).all() and (c.o[5:] == 77).all()
    c = mk()
    c.table[2, 1] = -7
    c.run()
    assert c.status.tolist() == [0, 0, 32, 32, 0]
    S.check(c, rows=[0, 1, 2, 5, 6])
    c = mk()
    c.group_off[0] = 1                                   # request 0 is in no group
    c.run()
    assert c.status.tolist()[0] == 2 and (c.o[0] == 77).all()
    c = mk()
    c.group_off[1] = 99                                  # beyond B
    c.run()
    assert all(s in (0, 2) for s in c.status.tolist())


def test_a_members_bad_offsets_leave_other_groups_alone():
    c = S.Case([60, 61, 90, 95], [1, 1, 1, 1], Hq=4, H=2, groups=[(0, 2, 30), (2, 4, 50)], seed=28)
    c.off[4] = 10 ** 6
    c.run()
    st = c.status.tolist()
    assert st[:2] == [0, 0] and st[2:] == [2, 2]
    S.check(c, rows=[0, 1])


@pytest.mark.parametrize("kind", _kinds(), ids=["window", "shared"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streams_graphs_and_repeats(kind, dtype):
    """The same bits again, on another stream, from two graphs that share nothing, and with two calls in flight."""
    a = S.Case([260, 2800, 275], [1, 20, 2], Hq=8, H=2, dtype=dtype, seed=30, **kind)
    b = S.Case([90, 1500, 300], [2, 1, 60], Hq=8, H=2, dtype=dtype, seed=31, **kind)
    want = []
    for c in (a, b):
        c.run()
        S.check(c)
        want.append((c.o.clone(), c.lse.clone()))
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [c.call(c.params()) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st, ws in zip((a, b), s, wss):
            c.o.fill_(1)
            st.wait_stream(torch.cuda.current_stream())
            c.call(c.params(), ws, st)
    torch.cuda.synchronize()
    for c, (o, lse) in zip((a, b), want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    graphs = []
    for c, ws in zip((a, b), wss):
        g = torch.cuda.CUDAGraph()
        p = c.params()
        with torch.cuda.graph(g):
            c.call(p, ws)
        graphs.append((g, p))
        c.o.fill_(2)
        c.lse.fill_(2)
    for _ in range(2):
        for (g, _), st in zip(graphs, s):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
    for c, (o, lse) in zip((a, b), want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("kind", ["window", "shared"])
def test_many_requests(kind):
    rng = np.random.default_rng(32)
    n = 700
    prefix = rng.integers(5, 40, n).tolist()
    sizes = rng.integers(1, 4, n).tolist()
    kw = dict(window=9, sinks=2) if kind == "window" else dict(groups=[(i, min(n, i + 3), 5) for i in range(0, n, 3)])
    c = S.Case(prefix, sizes, Hq=2, H=1, seed=33, **kw)
    c.run()
    S.check(c)


@pytest.mark.parametrize("members", [0, 1, 2])
def test_more_requests_than_a_kernels_start_holds(members):
    """Past 1024 entries and groups (1650 of groups of two, 2200 of one; 0: a window) costs and offsets are read again."""
    n = 1100
    prefix = np.random.default_rng(members).integers(5, 40, n).tolist()
    kw = dict(groups=[(i, i + members, 5) for i in range(0, n, members)]) if members else dict(window=9, sinks=2)
    c = S.Case(prefix, [1] * n, Hq=2, H=1, seed=35 + members, **kw)
    c.run()
    S.check(c)


def test_offsets_beyond_32_bits():
    """Pages at the far end of caches of more than 2^31 elements."""
    bs, H, d = 128, 8, 128
    nb = (1 << 31) // (bs * H * d) + 40
    for kw in (dict(window=200, sinks=3), dict(groups=[(0, 2, 150)])):
        c = S.Case([300, 310], [1, 2], Hq=8, H=H, bs=bs, seed=34, **kw)
        used = c.k.shape[0]
        k = torch.zeros((nb, H, bs, d), dtype=BF16, device="cuda")
        v = torch.zeros_like(k)
        k[nb - used:], v[nb - used:] = c.k, c.v
        table = torch.where(c.table >= 0, c.table + (nb - used), c.table)
        c.run(k_cache=k, v_cache=v, block_table=table)
        S.check(c)
        del k, v


# ------------------------------------------------------------------------------------ in a round
@pytest.mark.parametrize("kind", ["window", "shared"])
def test_verify_rounds(kind):
    """VerifyStep with a window as wide as the cache, and with groups whose prefixes are the same pages: the plain
    round's tokens; its twin, its graph and a narrow window run."""
    from speculative_decoding_draft_tree_gb300 import workloads as W
    from speculative_decoding_draft_tree_gb300.api import VerifyStep
    w = W.make_config(4, scale="small", device="cuda")
    if kind == "shared":      # every request's first pages become the first one's
        P = int(w.prefix_len.min())
        w.block_table[:, :P // w.k_cache.shape[3]] = w.block_table[0, :P // w.k_cache.shape[3]].clone()
    caches = (w.k_cache.clone(), w.v_cache.clone())
    plain = VerifyStep(w)
    plain.run()
    torch.cuda.synchronize()
    want = (plain.out_tokens.clone(), plain.out_len.clone(), plain.o.clone())

    def again():
        w.k_cache.copy_(caches[0])
        w.v_cache.copy_(caches[1])

    step = VerifyStep(w)
    if kind == "window":
        step.enable_window(1 << 20)
    else:
        P -= P % w.k_cache.shape[3]
        step.enable_shared(U.ints([0, w.B]), U.ints([P]))
    for s in (step, step.twin()):
        again()
        s.run()
        torch.cuda.synchronize()
        assert s.req_status.tolist() == [0] * w.B
        assert torch.equal(s.out_tokens, want[0]) and torch.equal(s.out_len, want[1])
        assert (s.o.double() - want[2].double()).norm() <= 6.4e-3 * want[2].double().norm()
    again()
    g = step.capture_graph()
    step.out_tokens.fill_(-5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(step.out_tokens, want[0])
    if kind == "window":
        again()
        narrow = VerifyStep(w)
        narrow.enable_window(40, 4)
        narrow.run()
        torch.cuda.synchronize()
        assert narrow.req_status.tolist() == [0] * w.B
        assert (narrow.o.double() - want[2].double()).norm() > 0.05 * want[2].double().norm()
    with pytest.raises(ValueError, match="do not combine"):
        step.enable_window(5)
