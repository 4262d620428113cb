"""GPU tests of data errors in the caches' operators: what has to be reported, and that nothing is
written for a request that is refused."""
import numpy as np
import pytest
import torch

import kv8_util as U
from speculative_decoding_draft_tree_gb300 import binding as B
from test_gpu_kv8 import AppendCase

pytestmark = pytest.mark.gpu


def _compact_case(late, T=200, Bn=24, bs=16, seed=0):
    """Paths of T - 1 steps that move every row but the first; each odd request's `late` steps read a
    page outside the pool (or, for "parent", step below their index)."""
    rng = np.random.default_rng(seed)
    prefix = rng.integers(0, 60, Bn).tolist()
    nodes = 2 * T
    need = [-(-(p + nodes) // bs) for p in prefix]
    nb = sum(need) + 2
    table = U.table_for(need, nb, rng)
    path = np.array([[0] + [d + 100 for d in range(1, T)] for _ in range(Bn)], dtype=np.int32)
    want = [0] * Bn
    for r in range(1, Bn, 2):
        if late == "page":
            want[r] = 32                                   # slots that only steps from 64 on read or write
            table[r, (prefix[r] + 100 + 64 + 5 * r) // bs + 1] = -1 if r % 4 == 1 else nb + 3
        else:
            want[r] = 1
            path[r, 64 + 5 * r % 100] = 3
    return prefix, table, path, nb, want


@pytest.mark.parametrize("late", ["page", "parent"])
def test_kv8_compact_refuses_a_late_bad_step_in_every_cta(late):
    """Long paths whose bad step lies in other warps' share, many layers and heads, so that many CTAs
    of a request check it while one of them reports it."""
    L, H, d, bs, T = 24, 16, 32, 16, 200
    prefix, table, path, nb, want = _compact_case(late, T)
    rng = np.random.default_rng(1)
    (k, ks), (v, vs) = [U.random_cache(L, nb, H, bs, d, rng) for _ in range(2)]
    before = [t.clone() for t in (k.view(torch.uint8), v.view(torch.uint8), ks, vs)]
    Bn = len(prefix)
    tab, pre, pth = torch.from_numpy(table).cuda(), U.ints(prefix), torch.from_numpy(path).cuda()
    n_acc = U.ints([T - 1] * Bn)
    bad = [r for r in range(Bn) if want[r]]
    pages = np.unique(np.concatenate([table[r][(table[r] >= 0) & (table[r] < nb)] for r in bad]))
    for _ in range(5):
        st, lens, used = (torch.zeros(Bn, dtype=torch.int32, device="cuda") for _ in range(3))
        moves = torch.zeros((Bn, T, 2), dtype=torch.int32, device="cuda")
        B.spec_kv8_compact(B.kv8_compact_params(k, v, ks, vs, tab, pre, pth, n_acc, st, lens, moves, used, T))
        torch.cuda.synchronize()
        assert st.cpu().tolist() == want
        assert lens.cpu().tolist() == [p if want[r] else p + T for r, p in enumerate(prefix)]
        assert (moves[bad] == -1).all()
        for t, b in zip((k.view(torch.uint8), v.view(torch.uint8), ks, vs), before):
            assert torch.equal(t[:, pages], b[:, pages])


@pytest.mark.parametrize("late", ["page", "parent"])
def test_kv_compact_refuses_a_late_bad_step_in_every_cta(late):
    """The same in the 16-bit cache."""
    L, H, d, bs, T = 48, 4, 32, 16, 200
    prefix, table, path, nb, want = _compact_case(late, T)
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn((L, nb, H, bs, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    before = (k.clone(), v.clone())
    Bn = len(prefix)
    tab, pre, pth = torch.from_numpy(table).cuda(), U.ints(prefix), torch.from_numpy(path).cuda()
    n_acc = U.ints([T - 1] * Bn)
    bad = [r for r in range(Bn) if want[r]]
    pages = np.unique(np.concatenate([table[r][(table[r] >= 0) & (table[r] < nb)] for r in bad]))
    for _ in range(5):
        st, lens, used = (torch.zeros(Bn, dtype=torch.int32, device="cuda") for _ in range(3))
        moves = torch.zeros((Bn, T, 2), dtype=torch.int32, device="cuda")
        B.spec_kv_compact(B.compact_params(k, v, tab, pre, pth, n_acc, st, lens, moves, used, T))
        torch.cuda.synchronize()
        assert st.cpu().tolist() == want
        assert lens.cpu().tolist() == [p if want[r] else p + T for r, p in enumerate(prefix)]
        assert (moves[bad] == -1).all()
        for t, b in zip((k, v), before):
            assert torch.equal(t[:, pages], b[:, pages])


def test_kv_compact_refuses_steps_past_32_bits():
    """P + path[d] beyond 2^31 - 1 is a bad step, in both caches."""
    L, H, d, bs, T = 2, 2, 32, 16, 4
    table = np.arange(16, dtype=np.int32).reshape(4, 4)
    path = np.array([[0, 2, 3, -1], [0, 2 ** 31 - 1, 3, -1], [0, 2 ** 31 - 20, 2 ** 31 - 20, -1], [0, 2, 3, -1]], dtype=np.int32)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn((L, 16, H, bs, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    rng = np.random.default_rng(4)
    (k8, ks), (v8, vs) = [U.random_cache(L, 16, H, bs, d, rng) for _ in range(2)]
    held = (torch.from_numpy(table).cuda(), U.ints([20, 20, 30, 1]), torch.from_numpy(path).cuda(), U.ints([2] * 4))
    for make, run, cache in ((lambda *a: B.compact_params(k, v, *a), B.spec_kv_compact, (k, v)),
                             (lambda *a: B.kv8_compact_params(k8, v8, ks, vs, *a), B.spec_kv8_compact, (k8.view(torch.uint8), v8.view(torch.uint8)))):
        before = [t.clone() for t in cache]
        st, lens, used = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3))
        moves = torch.zeros((4, T, 2), dtype=torch.int32, device="cuda")
        run(make(*held, st, lens, moves, used, T))
        torch.cuda.synchronize()
        assert st.cpu().tolist() == [0, 1, 1, 0] and lens.cpu().tolist() == [23, 20, 30, 4]
        for t, b in zip(cache, before):
            assert torch.equal(t[:, 4:12], b[:, 4:12]) and not torch.equal(t, b)


# ------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("off,start,want", [
    ([0, 18, 30], [0, 0], [0, 2]),                        # begins at N and ends past it
    ([0, 18, 25, 40], [3, 0, 0], [0, 2, 2]),
    ([0, 5, 3, 8, 18], [0, 7, 1, 20], [0, 2, 2, 0]),      # goes backwards; begins below an earlier offset
    ([6, 2, 2, 9, 18], [0, 0, 4, 1], [2, 2, 2, 0]),
    ([0, 12, 5, 14, 18], [0, 0, 0, 9], [0, 2, 2, 0]),
    ([-3, 0, 9, 18], [0, 2, 5], [2, 0, 0]),               # a negative offset without a row in [0, N)
    ([-9, -4, 6, 18], [0, 0, 1], [2, 2, 0]),
    ([0, 7, 7, 18, 18], [0, -1, 3, -8], [0, 2, 0, 2]),    # a negative start without rows
    ([0, 9, 18], [2 ** 31 - 9, 4], [2, 0]),               # slots past 32 bits
    ([18, 18, 18], [0, 0], [0, 0]),
])
@pytest.mark.parametrize("H", [2, 40])
def test_append_reports_every_request_that_cannot_be_appended(off, start, want, H):
    c = AppendCase([0] * len(start), [18] + [0] * (len(start) - 1), H=H, bs=4, seed=len(off), width=8, extra=40)
    rng = np.random.default_rng(3)
    c.table.copy_(torch.from_numpy(rng.permutation(c.nb)[:8 * len(start)].reshape(len(start), 8).astype(np.int32)))
    c.start, c.off = start, np.array(off)
    c.check()
    assert c.status.cpu().tolist() == want
    c.status.fill_(4)                                     # flagged by an earlier call: kept as it is
    c.check()
    assert c.status.cpu().tolist() == [4] * len(start)


@pytest.mark.parametrize("n", [3, 200])
def test_append_offsets_that_go_backwards_among_many_requests(n):
    """Several hundred requests and windows of several tokens; two stretches go backwards."""
    Bn, bs = 600, 16
    rng = np.random.default_rng(n)
    sizes = rng.integers(0, n, Bn)
    c = AppendCase(rng.integers(0, 40, Bn).tolist(), sizes.tolist(), H=1, d=32, bs=bs, seed=n)
    c.off[100] = c.off[103] + 2
    c.off[400:403] = c.off[390]
    c.check()
    st = c.status.cpu().numpy()
    assert (st == 2).sum() >= 3 and (st == 0).sum() > 500
