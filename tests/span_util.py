"""Inputs and comparisons of the GPU tests of windowed and shared-prefix attention."""
import numpy as np
import torch

import kv8_util as U
from oracle import span
from speculative_decoding_draft_tree_gb300 import binding as B


class Case:
    """One call over a random paged cache, and its oracle.  Slots that no row sees hold NaN, pages that no
    row sees are not in the table (-1)."""

    def __init__(self, prefix, sizes, Hq, H, d=128, bs=16, dtype=torch.bfloat16, window=None, sinks=0, groups=None,
                 T_max=None, seed=0, bits=None, q_scale=1.0, width=None, pad_rows=0, extra=3):
        rng = np.random.default_rng(seed)
        self.prefix, self.sizes, self.bs, self.window, self.sinks, self.groups = prefix, sizes, bs, window, sinks, groups
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
        self.N, self.off_np = int(off[-1]), off
        self.T_max = T_max or max(max(sizes), 1)
        self.bits = bits if bits is not None else [b for t in sizes for b in (U.chain_bits(t) if t < 17 else U.tree_bits(t, rng))]
        lengths = [0] * len(prefix)
        first = list(range(len(prefix)))
        for a, b, n in groups or []:
            for r in range(a, b):
                lengths[r], first[r] = n, a
        need = [-(-(p + t) // bs) for p, t in zip(prefix, sizes)]
        wide = width or max(max(need), 1)
        seen = [set(s for i in range(t) for s in span.visible(self.bits[off[r] + i], p, t, window, sinks)) for r, (p, t) in enumerate(zip(prefix, sizes))]
        pages = [sorted({s // bs for s in seen[r] if s // bs < wide}) for r in range(len(prefix))]
        nb = sum(len(p) for p in pages) + sum(need[a] for a, _, _ in groups or []) + extra
        ids = list(rng.permutation(nb))
        table = np.full((len(prefix), wide), -1, dtype=np.int32)
        live = np.zeros((nb, bs), dtype=bool)
        for r in range(len(prefix)):
            leads = first[r] == r and lengths[r] > 0
            for p in pages[r]:
                if p * bs + bs > lengths[r] or leads:
                    table[r, p] = ids.pop()
        for r in range(len(prefix)):
            for s in seen[r]:
                if s // bs < wide:
                    live[table[first[r] if s < lengths[r] else r, s // bs], s % bs] = True
        g = torch.Generator(device="cuda").manual_seed(seed + 7)
        rows = self.N + pad_rows
        dead = torch.from_numpy(~live).cuda()[:, None, :, None]
        mag = torch.exp2(torch.rand((H, 1, 1), generator=g, device="cuda") * 2 - 1)
        self.k, self.v = [(torch.randn((nb, H, bs, d), generator=g, device="cuda") * mag).to(dtype).masked_fill_(dead, float("nan")) for _ in range(2)]
        self.q = (torch.randn((rows, Hq, d), generator=g, device="cuda") * q_scale).to(dtype)
        self.anc = U.mask_words(self.bits + [1] * pad_rows, self.T_max)
        self.table_np, self.table = table, torch.from_numpy(table).cuda()
        self.prefix_t, self.off = U.ints(prefix), U.ints(off.tolist())
        self.status = torch.zeros(len(prefix), dtype=torch.int32, device="cuda")
        self.o = torch.full_like(self.q, 77.0)
        self.lse = torch.full((rows, Hq), 55.0, dtype=torch.float32, device="cuda")
        if groups is not None:
            self.group_off, self.shared = U.ints([a for a, _, _ in groups] + [groups[-1][1]]), U.ints([n for _, _, n in groups])

    def params(self, **kw):
        a = dict(q=self.q, k_cache=self.k, v_cache=self.v, block_table=self.table, prefix_len=self.prefix_t, node_offset=self.off,
                 anc_mask=self.anc, T_max=self.T_max, o=self.o, lse=self.lse, req_status=self.status)
        if self.groups is None:
            a.update(window=self.window, sinks=self.sinks)
        else:
            a.update(group_offset=self.group_off, shared_len=self.shared)
        a.update(kw)
        return (B.attention_window_params if self.groups is None else B.attention_shared_params)(**a)

    def call(self, p, ws=None, stream=None):
        size, run = ((B.spec_attention_window_workspace_size, B.spec_tree_attention_window) if self.groups is None
                     else (B.spec_attention_shared_workspace_size, B.spec_tree_attention_shared))
        if ws is None:
            ws = torch.full((max(256, size(p)),), 0xA5, dtype=torch.uint8, device="cuda")
        run(p, ws, stream)
        return ws

    def run(self, stream=None, **kw):
        self.call(self.params(**kw), None, stream)
        torch.cuda.synchronize()
        return self.o, self.lse

    def oracle(self, scale=None):
        val = lambda t: torch.nan_to_num(t.double(), nan=0.0).cpu().numpy()  # noqa: E731
        return span.attention(self.q[:self.N].double().cpu().numpy(), val(self.k), val(self.v), self.table_np, self.prefix, self.off_np,
                              self.bits, self.bs, scale, self.window, self.sinks, self.groups)


def check(case, rows=None, scale=None):
    """Bars by arithmetic, elementwise.

    Scores: the products of bf16 (or fp32) elements are summed in fp32; 2^-17 of the sum of their magnitudes
    covers 128 .. 256 roundings of 2^-24 and the tensor core's truncations.  E is that for a row's key with the
    largest sum, plus 2^-20 for the exponential (2^-22) and the sums of weights: a weight is off by a factor
    within e^E, a ratio of sums within e^2E.
    Weights: bf16 products take them as bf16 (off by at most half a step, 2^-8 of themselves) or as two bf16
    pieces (2^-16).  Which of both a row gets depends on how many rows lie beside it: 2^-8 holds for both.
    Output: one rounding, bf16 2^-8, fp32 2^-24 (2^-17 with the sums over the row).
    All outputs together: each rounding is even within its half step, so the root mean square of one is at most
    2^-8 / sqrt(3) = 0.00226 of the values, of two 0.0032.
    """
    o, lse, mass, size = case.oracle(scale)
    go, gl = case.o[:case.N].double().cpu().numpy(), case.lse[:case.N].double().cpu().numpy()
    f32 = case.q.dtype == torch.float32
    E = 2.0 ** -17 * size + 2.0 ** -20
    tol = (2 * E[..., None] + (0 if f32 else 2.0 ** -8)) * mass + (2.0 ** -17 * mass if f32 else 2.0 ** -8 * np.abs(o))
    sel = slice(None) if rows is None else rows
    bad = ~(np.abs(go - o)[sel] <= tol[sel] + 1e-30)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(go - o)[sel])))
    seen = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(gl)[sel], ~seen[sel])
    assert (go[sel][~seen[sel]] == 0).all()
    ltol = E + 2.0 ** -21 * np.abs(np.where(seen, lse, 0)) + 2.0 ** -19
    assert (np.abs(np.where(seen, gl - np.where(seen, lse, 0), 0)) <= ltol)[sel].all()
    norm = np.linalg.norm(o[sel])
    if norm > 0:
        assert np.linalg.norm((go - o)[sel]) <= (3.2e-3 if not f32 else 2e-5) * norm
    return o, lse
