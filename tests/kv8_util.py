"""Inputs and comparisons of the 8-bit cache's GPU tests."""
import numpy as np
import torch

from oracle import kv8 as K
from speculative_decoding_draft_tree_gb300 import binding as B

E4M3 = torch.float8_e4m3fn


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def values(codes):
    """The values of a code tensor (float8 or its bytes) as float64 numpy."""
    return codes.view(E4M3).double().cpu().numpy()


def table_for(need, num_blocks, rng, width=None):
    """Distinct random pages for each request; -1 past its need."""
    ids = rng.permutation(num_blocks)
    t = np.full((len(need), width or max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        n = min(n, t.shape[1])
        t[r, :n] = ids[at:at + n]
        at += n
    assert at <= num_blocks
    return t


def random_cache(L, nb, H, bs, d, rng, spread=4, junk=True):
    """Codes and power-of-two scales as tensors [L, nb, H, bs, d], [L, nb, H]; with `junk` the
    codes include every bit pattern but NaN."""
    c = rng.integers(0, 256, (L, nb, H, bs, d)).astype(np.uint8)
    if not junk:
        x = rng.normal(size=(L, nb, H, bs, d)) * 90
        return (torch.from_numpy(K.round_e4m3(x)).to(E4M3).cuda(),
                torch.from_numpy(2.0 ** rng.integers(-9, -9 + spread, (L, nb, H))).float().cuda())
    c[(c & 127) == 127] = 3
    s = 2.0 ** rng.integers(-9, -9 + spread, (L, nb, H))
    return torch.from_numpy(c).cuda().view(E4M3), torch.from_numpy(s).float().cuda()


def chain_bits(T):
    return [(1 << (i + 1)) - 1 for i in range(T)]


def tree_bits(T, rng):
    out = []
    for i in range(T):
        p = -1 if i == 0 else int(rng.integers(max(0, (i - 1) // 3), i))
        out.append((out[p] if p >= 0 else 0) | (1 << i))
    return out


def mask_words(bits, T_max):
    W = (T_max + 31) // 32
    w = np.array([[(b >> (32 * j)) & 0xFFFFFFFF for j in range(W)] for b in bits], dtype=np.uint32).reshape(len(bits), W)
    return torch.from_numpy(w.view(np.int32)).cuda()


class AttnCase:
    """Inputs of one attention call over a random 8-bit cache, and its oracle.  Codes and scales of
    everything that is not live are poisoned (NaN codes, NaN scales in dead blocks)."""

    def __init__(self, prefix, sizes, Hq, H, d=128, bs=16, dtype=torch.bfloat16, T_max=None, seed=0, bits=None,
                 q_scale=1.0, spread=4, width=None, pad_rows=0, poison=True):
        rng = np.random.default_rng(seed)
        self.prefix, self.sizes, self.bs, self.d = prefix, sizes, bs, d
        need = [-(-(p + t) // bs) for p, t in zip(prefix, sizes)]
        nb = sum(need) + 3
        self.table_np = table_for(need, nb, rng, width)
        k, ks = random_cache(1, nb, H, bs, d, rng, spread, junk=False)
        v, vs = random_cache(1, nb, H, bs, d, rng, spread, junk=False)
        self.k, self.ks, self.v, self.vs = k[0], ks[0], v[0], vs[0]
        if poison:
            live = torch.zeros((nb, bs), dtype=torch.bool)
            for r, (p, t) in enumerate(zip(prefix, sizes)):
                for s in range(p + t):
                    live[int(self.table_np[r][s // bs]), s % bs] = True
            dead = ~live.cuda()
            for c in (self.k, self.v):
                c.view(torch.uint8).masked_fill_(dead[:, None, :, None], 0x7F)
            blocks = dead.all(dim=1)
            self.ks[blocks] = float("nan")
            self.vs[blocks] = float("inf")
        off = np.concatenate([[0], np.cumsum(sizes)]).astype(int)
        self.N = int(off[-1])
        self.T_max = T_max or max(max(sizes), 1)
        self.bits = bits if bits is not None else [b for t in sizes for b in (chain_bits(t) if t < 17 else tree_bits(t, rng))]
        g = torch.Generator(device="cuda").manual_seed(seed + 7)
        rows = self.N + pad_rows
        self.q = (torch.randn((rows, Hq, d), generator=g, device="cuda") * q_scale).to(dtype)
        self.anc = mask_words(self.bits + [1] * pad_rows, self.T_max)
        self.table, self.off_np = torch.from_numpy(self.table_np).cuda(), off
        self.prefix_t, self.off = ints(prefix), ints(off.tolist())
        self.status = torch.zeros(len(prefix), dtype=torch.int32, device="cuda")
        self.o = torch.full_like(self.q, 77.0)
        self.lse = torch.full((rows, Hq), 55.0, dtype=torch.float32, device="cuda")

    def params(self, **kw):
        a = dict(q=self.q, k_cache=self.k, v_cache=self.v, k_scale=self.ks, v_scale=self.vs, block_table=self.table,
                 prefix_len=self.prefix_t, node_offset=self.off, anc_mask=self.anc, T_max=self.T_max, o=self.o,
                 lse=self.lse, req_status=self.status)
        a.update(kw)
        return B.attention_kv8_params(**a)

    def run(self, stream=None, **kw):
        p = self.params(**kw)
        ws = torch.full((max(256, B.spec_attention_kv8_workspace_size(p)),), 0xA5, dtype=torch.uint8, device="cuda")
        B.spec_tree_attention_kv8(p, ws, stream)
        torch.cuda.synchronize()
        return self.o, self.lse

    def oracle(self, scale=None):
        vis = [[(b >> j) & 1 for j in range(self.T_max)] for b in self.bits]
        return K.tree_attention(self.q[:self.N].double().cpu().numpy(), np.nan_to_num(values(self.k)),
                                np.nan_to_num(self.ks.double().cpu().numpy(), posinf=0.0), np.nan_to_num(values(self.v)),
                                np.nan_to_num(self.vs.double().cpu().numpy(), posinf=0.0), self.table_np, self.prefix,
                                self.off_np, vis, self.bs, scale)


def check_attention(case, rows=None, scale=None):
    """Bars by arithmetic, elementwise.

    Scores: bf16 queries enter the products as two e4m3 pieces, off by at most 2^-10 of a range in
    which the row's largest element is above 224: 2^-17.8 max|q| for each element; the products are
    exact and summed in fp32 (2^-17 of the sum of their magnitudes covers the tensor core's sums).  E is
    the sum of both: a weight is off by a factor within e^E.
    Weights, units of at most 16 query rows: 11-bit halves split into two e4m3 pieces, each rounded to
    within 2^-4 of itself, so off by 2^-8 + 2^-11 of themselves or (where the second piece is
    subnormal) by 2^-10 of a range in which a row's largest weight is at least 2^6: 2^-16 of the largest.
    Longer units: the first piece is e5m2, rounded to within 2^-3 of the weight, so the second, e4m3 of
    that remainder, leaves 2^-4 2^-3 = 2^-7 (and the halves' 2^-11), or 2^-10 of a range in which a
    row's largest weight is at least 2^3: 2^-13 of the largest.
    Output: that, and one rounding to bf16 (2^-8 of the value).  fp32 queries take the CUDA-core
    kernel: fp32 products and sums over the row (2^-17 relative bounds them), exp2 within 2^-21.
    """
    o, lse, mass, err, tail = case.oracle(scale)
    go = case.o[:case.N].double().cpu().numpy()
    gl = case.lse[:case.N].double().cpu().numpy()
    f32 = case.q.dtype == torch.float32
    E = (0.0 if f32 else 2.0 ** -17.8) * err[..., 0] + 2.0 ** -17 * err[..., 1] + 2.0 ** -20
    if f32:
        tol = 2 * E[..., None] * mass + 2.0 ** -17 * mass
    else:
        few = case.T_max * (case.q.shape[1] // case.ks.shape[1]) <= 16
        rel, least = (2.0 ** -8, 2.0 ** -16) if few else (2.0 ** -7, 2.0 ** -13)
        tol = (2 * E[..., None] + rel + 2.0 ** -11) * mass + least * tail + 2.0 ** -8 * np.abs(o)
    sel = slice(None) if rows is None else rows
    bad = np.abs(go - o)[sel] > tol[sel] + 1e-30
    assert not bad.any(), (int(bad.sum()), float(np.abs(go - o).max()))
    seen = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(gl)[sel], ~seen[sel])
    assert (go[~seen] == 0).all()
    ltol = E + 2.0 ** -21 * np.abs(np.where(seen, lse, 0)) + 2.0 ** -19
    assert (np.abs(np.where(seen, gl - np.where(seen, lse, 0), 0)) <= ltol)[sel].all()
    norm = np.linalg.norm(o[sel])
    if norm > 0:   # and over all outputs: the roundings do not add up one way
        assert np.linalg.norm((go - o)[sel]) <= (3e-3 if not f32 else 2e-5) * norm
    return o, lse
