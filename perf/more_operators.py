"""Operators of long and of many continuations over the paged K/V cache: cases, inputs, plain forms
and exact values.

  shared   tree attention for groups of requests that continue one prompt: the prompt's keys and values
           are read once for all of a group's rows, each request's own ones for its own rows
  window   tree attention with a sliding window and a few first tokens (sinks) that stay visible; pages
           that no row can see any more may have been given back, their table entries are -1
  select   beam search: the best W of W x V continuations of each request, finished beams kept
  reorder  the beams' cache follows the selection: tables inherit the parents' full pages, the page that
           is being written is kept by a parent's first child and copied for its other children

`run` computes the plain form with elementary torch operations, or, where `own` is true, makes
the calls a user of the framework makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases
def listed():
    return [
        # four beams of one prompt, a few tokens in: latency counts
        dict(name="shared 4 beams x 509", op="shared", groups=1, members=4, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", bs=16, shared=509, lo=3, hi=21, paged="scattered"),
        # eight samples for each of eight prompts
        dict(name="shared 8 x 8 samples", op="shared", groups=8, members=8, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", bs=16, shared=8192, lo=1, hi=511, paged="scattered"),
        # a decoding batch under one long common prompt, own parts of very different lengths
        dict(name="shared 64 under 32K", op="shared", groups=1, members=64, T=1, Hq=64, Hkv=8, D=128, dtype="bf16", bs=16, shared=32768, lo=1, hi=2048, paged="scattered"),
        # draft trees of a batch under one common prompt
        dict(name="shared 32 trees under 8K", op="shared", groups=1, members=32, T=46, Hq=32, Hkv=8, D=128, dtype="bf16", bs=16, shared=8192, lo=64, hi=1024, paged="runs"),
        # one request's next token, a window that is shorter than its cache: latency counts
        dict(name="window 1 token x 1024", op="window", B=1, T=1, Hq=32, Hkv=8, D=128, dtype="bf16", bs=16, lo=5000, hi=5000, window=1024, sinks=4, paged="scattered"),
        # a decoding batch with caches of very different lengths
        dict(name="window 64 ragged x 4096", op="window", B=64, T=1, Hq=64, Hkv=8, D=128, dtype="bf16", bs=16, lo=1024, hi=32768, window=4096, sinks=4, paged="scattered"),
        # fixed expansion trees of 46 tokens over long caches
        dict(name="window 32 trees x 2048", op="window", B=32, T=46, Hq=32, Hkv=8, D=128, dtype="bf16", bs=16, lo=3000, hi=8192, window=2048, sinks=64, paged="scattered"),
        # one request's four beams
        dict(name="select 1 x 4 of 32000", op="select", B=1, W=4, V=32000, dtype="bf16", alpha=0.0, tau=1.0),
        # a large vocabulary in 32 bits, length penalty
        dict(name="select 16 x 5 of 128256", op="select", B=16, W=5, V=128256, dtype="f32", alpha=0.6, tau=0.8),
        # the largest batch and vocabulary
        dict(name="select 64 x 8 of 152064", op="select", B=64, W=8, V=152064, dtype="bf16", alpha=1.0, tau=1.0),
        # one request's four beams, one layer
        dict(name="reorder 1 x 4, 1 layer", op="reorder", B=1, W=4, Hkv=8, D=128, bs=16, L=1, lo=137, hi=137, dtype="bf16"),
        # a batch's beams over a whole model's layers
        dict(name="reorder 32 x 8, 32 layers", op="reorder", B=32, W=8, Hkv=8, D=128, bs=32, L=32, lo=200, hi=900, dtype="bf16"),
    ]


def draw(rng):
    op = rng.choice(["shared", "shared", "window", "window", "select", "reorder"])
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    if op in ("shared", "window"):
        small = rng.random() < 0.15                       # the fp32 workloads are small
        T = rng.choice([1, 1, log(2, 16), log(17, 100)])
        Hkv = rng.choice([1, 2, 4]) if small else rng.choice([1, 2, 4, 8, 8, 16])
        G = rng.choice([1, 2, 4]) if small else rng.choice([1, 2, 4, 5, 7, 8, 16])
        D, dtype = (rng.choice([64, 128]), "f32") if small else (128, "bf16")
        bs = rng.choice([16, 16, 32, 64])
        hi = log(16, 600 if small else 32768)
        shape = dict(op=op, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, dtype=dtype, bs=bs, paged=rng.choice(["scattered", "runs"]))
        # no dearer than the largest listed case: sum of T * Hq * keys and of Hkv * keys
        most = min(64, 64 * 8 * 33000 // (Hkv * hi), 32 * 46 * 32 * 9000 // (T * G * Hkv * hi)) if not small else 4
        B = log(1, max(1, most))
        if op == "window":
            return dict(shape, B=B, lo=max(0, hi // rng.choice([1, 2, 16])), hi=hi, window=log(1, 8192), sinks=rng.choice([0, 1, 4, 64, 200]))
        groups = log(1, B)
        shared = hi if rng.random() < 0.8 else 0
        own_hi = log(1, max(1, hi // 4))
        return dict(shape, groups=groups, members=max(1, B // groups), shared=shared, lo=max(0, own_hi // rng.choice([1, 4, 64]) - 1), hi=own_hi)
    if op == "select":
        W, V = rng.randint(1, 16), log(50, 152064)
        return dict(op=op, B=log(1, max(1, min(128, 64 * 8 * 152064 // (2 * W * V)))), W=W, V=V, dtype=rng.choice(["bf16", "bf16", "f32"]), alpha=rng.choice([0.0, 0.6, 1.0]), tau=rng.choice([1.0, 1.0, 0.7, 1.3]))
    W = rng.randint(1, 12)
    return dict(op=op, B=log(1, 24), W=W, Hkv=rng.choice([1, 4, 8]), D=rng.choice([64, 128]), bs=rng.choice([16, 32, 64]), L=log(1, 32), lo=rng.randint(1, 90), hi=rng.randint(91, 900), dtype=rng.choice(["bf16", "bf16", "f32", "e4m3"]))


def _spread(n, lo, hi, salt):
    """n whole numbers over [lo, hi] in a mixed order; a case's sizes do not go by the seed."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 37 + salt) % n) // (n - 1) for i in range(n)]


def _lengths(case):
    """(cached tokens, new tokens) of each request of an attention case."""
    if case["op"] == "shared":
        B = case["groups"] * case["members"]
        prefix = [case["shared"] + p for p in _spread(B, case["lo"], case["hi"], 5)]
    else:
        B = case["B"]
        prefix = _spread(B, case["lo"], case["hi"], 5)
    T = case["T"]
    return prefix, [T] * B if T <= 16 else _spread(B, max(17, T // 2), T, 11)


def _live(case, P):
    """The slots below P that some row of a windowed request can see: [0, a) and [b, P)."""
    b = max(0, P - case["window"] + 1)
    return min(case["sinks"], b), b


def work(case):
    op = case["op"]
    if op in ("shared", "window"):
        prefix, new = _lengths(case)
        H, Hq, D, N = case["Hkv"], case["Hq"], case["D"], sum(new)
        es = 2 if case["dtype"] == "bf16" else 4
        if op == "shared":
            keys = case["groups"] * case["shared"] + sum(p - case["shared"] + t for p, t in zip(prefix, new))
            seen = sum(t * (p + 1) for p, t in zip(prefix, new))       # the prefix and itself at least
        else:
            live = [(_live(case, p), p) for p in prefix]
            keys = sum(a + p - b + t for ((a, b), p), t in zip(live, new))
            seen = sum(t * min(case["window"] + case["sinks"], p + 1) for p, t in zip(prefix, new))
        return {"bytes": 2 * keys * H * D * es + N * Hq * (2 * D * es + 4), "flops": 4 * seen * Hq * D}
    if op == "select":
        rows = case["B"] * case["W"]
        return {"bytes": rows * case["V"] * (2 if case["dtype"] == "bf16" else 4) + 40 * rows, "flops": 4 * rows * case["V"]}
    es = {"bf16": 2, "f32": 4, "e4m3": 1}[case["dtype"]]
    moved = 0
    for b, n in enumerate(_spread(case["B"], case["lo"], case["hi"], 5)):
        moved += (n % case["bs"]) * (case["W"] - len(set(_parents(case, b, 0))))
    return {"bytes": 2 * 2 * moved * case["L"] * case["Hkv"] * case["D"] * es + 8 * case["B"] * case["W"], "flops": 0}


def _parents(case, b, seed):
    """A request's parents as a selection leaves them: a few beams have most of the children. The number
    of different parents does not go by the seed."""
    W = case["W"]
    keep = max(1, (W * (2 + (b * 7) % 4) + 4) // 6)
    kept = [(i * 5 + b + seed) % W for i in range(W)]
    kept = list(dict.fromkeys(kept + list(range(W))))[:keep]
    return [kept[(i * i + b) % keep] if i >= keep else kept[i] for i in range(W)]


# --------------------------------------------------------------------------------------- inputs
def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _trees(new, seed):
    """Each request's tree: the ancestors-or-self of each node, as bits [N, words]."""
    import random
    rng = random.Random(seed)
    W = (max(new) + 31) // 32
    rows = []
    for T in new:
        anc = []
        for i in range(T):
            parent = i - 1 if T <= 16 else -1 if i == 0 else rng.randrange(max(0, (i - 1) // 3), i)
            anc.append((anc[parent] if parent >= 0 else 0) | (1 << i))
        rows += anc
    words = [[(b >> (32 * w)) & 0xFFFFFFFF for w in range(W)] for b in rows]
    return torch.tensor(words, dtype=torch.int64).to(torch.int32).cuda()


def _page_lists(case, prefix, new, seed):
    """Each request's pages as indices into the pool (-1: given back), and the pool's size."""
    bs, at, table = case["bs"], 0, []
    if case["op"] == "shared":
        full = case["shared"] // bs
        for r, (p, t) in enumerate(zip(prefix, new)):
            if r % case["members"] == 0:
                common = list(range(at, at + full))
                at += full
            n = -(-(p + t) // bs) - full
            table.append(common + list(range(at, at + n)))
            at += n
    else:
        for p, t in zip(prefix, new):
            a, b = _live(case, p)
            row = []
            for i in range(-(-(p + t) // bs)):
                if i * bs < a or (i + 1) * bs > b:
                    row.append(at)
                    at += 1
                else:
                    row.append(-1)
            table.append(row)
    size = at + max(1, at // 10)
    if case["paged"] == "scattered":
        ids = torch.randperm(size, generator=torch.Generator().manual_seed(seed)).tolist()
        table = [[ids[i] if i >= 0 else -1 for i in row] for row in table]
    wide = max(len(row) for row in table)
    return [row + [-1] * (wide - len(row)) for row in table], size


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "select":
        B, W, V = case["B"], case["W"], case["V"]
        logits = torch.randn((B * W, V), generator=g, device="cuda") * 3
        # a few likely tokens in each row, more so in some; one that comes up twice has the larger value, so
        # that the inputs go by the seed alone
        top = torch.randint(0, V, (B * W, min(V, 12)), generator=g, device="cuda")
        logits.scatter_reduce_(1, top, 8 + 6 * torch.rand(top.shape, generator=g, device="cuda"), "amax", include_self=False)
        ld = -(-V // 8) * 8
        rows = torch.zeros((B * W, ld), dtype=DTYPES[case["dtype"]], device="cuda")
        rows[:, :V] = logits.to(rows.dtype)
        steps = torch.rand((B, W), generator=g, device="cuda").cumsum(1) * 1.5
        length = 2 + torch.randint(0, 60, (B, 1), generator=g, device="cuda") + torch.zeros((B, W), dtype=torch.int64, device="cuda")
        finished = (torch.rand((B, W), generator=g, device="cuda") < 0.15).to(torch.int32)
        length = (length - finished * torch.randint(0, 2, (B, W), generator=g, device="cuda")).clamp(min=1)
        s = dict(op=op, B=B, W=W, V=V, tau=case["tau"], alpha=case["alpha"], eos=2 % V, rows=rows, score=-(steps + 0.8 * length.float()), length=length.to(torch.int32), finished=finished)
        for k, t in (("parent", torch.int32), ("token", torch.int32), ("new_score", torch.float32), ("new_length", torch.int32), ("new_finished", torch.int32)):
            s[k] = torch.empty((B, W), dtype=t, device="cuda")
    elif op == "reorder":
        B, W, bs, L, H, D = (case[k] for k in ("B", "W", "bs", "L", "Hkv", "D"))
        lens = _spread(B, case["lo"], case["hi"], 5)
        wide = max(lens) // bs + 3
        nb = B * W * 3 + 16          # the page written now and two more of each beam; full pages lie anywhere
        ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        table = ids[torch.randint(0, nb, (B * W, wide), generator=g, device="cuda")]
        at = torch.arange(B * W, device="cuda")
        page = torch.tensor(lens, device="cuda").repeat_interleave(W) // bs
        for k in range(3):
            table[at, (page + k).clamp(max=wide - 1)] = ids[k * B * W:(k + 1) * B * W]
        s = dict(op=op, B=B, W=W, bs=bs, table=table.contiguous(), kv_len=_ints(lens), status=torch.zeros(B, dtype=torch.int32, device="cuda"))
        s["parent"] = _ints([_parents(case, b, seed) for b in range(B)])
        shape = (L, nb, H, bs, D)
        if case["dtype"] == "e4m3":
            for k in ("k", "v"):
                s[k] = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
                s[k + "s"] = torch.exp2(torch.randint(-8, 3, shape[:3], generator=g, device="cuda").float())
        else:
            for k in ("k", "v"):
                s[k], s[k + "s"] = torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["dtype"]]), None
    else:
        prefix, new = _lengths(case)
        H, Hq, D, bs, dt = case["Hkv"], case["Hq"], case["D"], case["bs"], DTYPES[case["dtype"]]
        offset = [0]
        for n in new:
            offset.append(offset[-1] + n)
        N, B = offset[-1], len(new)
        pages, nb = _page_lists(case, prefix, new, seed)
        s = dict(op=op, bs=bs, prefix=_ints(prefix), offset=_ints(offset), table=_ints(pages), T_max=max(new), status=torch.zeros(B, dtype=torch.int32, device="cuda"))
        # heads have magnitudes of their own; queries lean toward a direction of each head, along which
        # the first tokens' keys are large
        lean = torch.randn((H, D), generator=g, device="cuda") / math.sqrt(D)
        head = torch.exp2(torch.rand((H, 1, 1), generator=g, device="cuda") - 0.5)
        q = torch.randn((N, H, Hq // H, D), generator=g, device="cuda") * 1.2 + 4 * lean[:, None]
        s["q"] = q.reshape(N, Hq, D).to(dt)
        s["k"] = torch.empty((nb, H, bs, D), dtype=dt, device="cuda")
        s["v"] = torch.empty((nb, H, bs, D), dtype=dt, device="cuda")
        step = max(1, (64 << 20) // (H * bs * D))
        for b in range(0, nb, step):
            n = min(step, nb - b)
            s["k"][b:b + n] = (torch.randn((n, H, bs, D), generator=g, device="cuda") * head).to(dt)
            s["v"][b:b + n] = torch.randn((n, H, bs, D), generator=g, device="cuda").to(dt)
        for r in range(B):
            if prefix[r] > 0 and pages[r][0] >= 0 and (op == "window" or r % case["members"] == 0):
                s["k"][pages[r][0], :, 0] = (8 * lean).to(dt)
        if op == "window":
            s["window"], s["sinks"] = case["window"], case["sinks"]
        else:
            m, shared = case["members"], case["shared"]
            s["group"], s["shared"] = _ints(list(range(0, B + 1, m))), _ints([shared] * case["groups"])
            if shared % bs:          # the forks copied the rows of the prompt's last page
                for r in range(B):
                    a, b = pages[r - r % m][shared // bs], pages[r][shared // bs]
                    for cache in (s["k"], s["v"]):
                        cache[b, :, :shared % bs] = cache[a, :, :shared % bs]
        s["mask"] = _trees(new, seed)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((N, Hq), dtype=torch.float32, device="cuda")
        s["req"] = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"))
        s["node"] = torch.arange(N, device="cuda") - s["offset"][:-1].long()[s["req"]]
    if own:
        s["plan"] = _plan(s)
    return s


def _plan(s):
    """The parameter block and the workspace that a user's program keeps."""
    from speculative_decoding_draft_tree_gb300 import binding as K
    if s["op"] == "shared":
        p = K.attention_shared_params(s["q"], s["k"], s["v"], s["table"], s["prefix"], s["offset"], s["mask"], s["T_max"], s["group"], s["shared"], s["o"], s["lse"], s["status"])
        size = K.spec_attention_shared_workspace_size(p)
    elif s["op"] == "window":
        p = K.attention_window_params(s["q"], s["k"], s["v"], s["table"], s["prefix"], s["offset"], s["mask"], s["T_max"], s["window"], s["sinks"], s["o"], s["lse"], s["status"])
        size = K.spec_attention_window_workspace_size(p)
    elif s["op"] == "select":
        p = K.beam_select_params(s["rows"], s["V"], s["tau"], s["score"], s["length"], s["finished"], s["eos"], s["alpha"], s["parent"], s["token"], s["new_score"], s["new_length"], s["new_finished"])
        size = K.spec_beam_select_workspace_size(p)
    else:
        p = K.beam_reorder_params(s["k"], s["v"], s["table"], s["kv_len"], s["parent"], s["status"], s["ks"], s["vs"])
        size = K.spec_beam_reorder_workspace_size(p)
    return p, torch.empty(max(256, size), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------------- plain forms
def run(s):
    if own:
        return _run_own(s)
    return {"shared": _attend, "window": _attend, "select": _select, "reorder": _reorder}[s["op"]](s)


def _run_own(s):
    from speculative_decoding_draft_tree_gb300 import binding as K
    if s["op"] == "shared":
        K.spec_tree_attention_shared(*s["plan"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "window":
        K.spec_tree_attention_window(*s["plan"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "select":
        K.spec_beam_select(*s["plan"])
        return {k: s[k] for k in ("parent", "token", "new_score", "new_length", "new_finished")}
    K.spec_beam_reorder(*s["plan"])
    return {k: s[k] for k in ("k", "v", "ks", "vs", "table") if s[k] is not None}


def _depth(mask):
    """The depth of each node: how many ancestors its bits name."""
    bits = (mask[:, :, None] >> torch.arange(32, dtype=torch.int32, device="cuda")) & 1
    return bits.sum(dim=(1, 2)) - 1


def _visible(s, S):
    """[N, S]: whether a node sees a slot of its request."""
    slot = torch.arange(S, device="cuda")
    req, words = s["req"], s["mask"].shape[1]
    P = s["prefix"].long()[req][:, None]
    a = slot[None, :] - P                                             # tree index of a slot
    word = s["mask"].gather(1, (a >> 5).clamp(0, words - 1))
    seen = ((word >> (a & 31).to(torch.int32)) & 1).bool()
    count = (s["offset"][1:] - s["offset"][:-1]).long()[req][:, None]
    inside = (a >= 0) & (a < count)
    if s["op"] == "shared":
        return (a < 0) | (seen & inside)
    depth = _depth(s["mask"])
    at = (s["offset"][:-1].long()[req][:, None] + a).clamp(0, depth.numel() - 1)
    pos = torch.where(a < 0, slot[None, :], P + depth[at])            # position of a slot
    near = ((P + depth[:, None]) - pos < s["window"]) | (pos < s["sinks"])
    return ((a < 0) | (seen & inside)) & near


def _attend(s):
    q, table, bs = s["q"].float(), s["table"].long().clamp(min=0), s["bs"]
    N, Hq, D = q.shape
    B, nblk = table.shape
    H, S, T = s["k"].shape[1], nblk * bs, s["T_max"]
    G = Hq // H
    gather = lambda cache: cache[table.view(-1)].float().view(B, nblk, H, bs, D).transpose(1, 2).reshape(B, H, S, D)  # noqa: E731
    qp = torch.zeros((B, T, Hq, D), device="cuda")
    qp[s["req"], s["node"]] = q
    rows = qp.view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    x = torch.matmul(rows, gather(s["k"]).transpose(2, 3)) * (1.0 / math.sqrt(D))
    vis = torch.zeros((B, T, S), dtype=torch.bool, device="cuda")
    vis[s["req"], s["node"]] = _visible(s, S)
    x.view(B, H, T, G, S).masked_fill_(~vis[:, None, :, None, :], -math.inf)
    m = x.amax(dim=-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    x.sub_(m).exp_()
    total = x.sum(dim=-1, keepdim=True)
    o = torch.matmul(x, gather(s["v"])) / torch.where(total > 0, total, torch.ones_like(total))
    back = lambda t: t.view(B, H, T, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, -1)[s["req"], s["node"]]  # noqa: E731
    return {"o": back(o).to(s["q"].dtype), "lse": back(m + total.log())[..., 0]}


def _penalty(length, alpha):
    return ((5.0 + length.double()) / 6.0) ** alpha


def _select(s):
    """Scores next to one another decide, so their sums are taken in 64 bits."""
    B, W, V = s["B"], s["W"], s["V"]
    x = s["rows"][:, :V].double() / s["tau"]
    m = x.amax(dim=1, keepdim=True)
    logp = x - (m + (x - m).exp().sum(dim=1, keepdim=True).log())
    score, done, length = s["score"].double(), s["finished"].bool(), s["length"]
    total = score[:, :, None] + logp.view(B, W, V)
    keep = torch.full((1, 1, V), -math.inf, dtype=torch.float64, device="cuda")
    keep[0, 0, s["eos"]] = 0
    total = torch.where(done[:, :, None], score[:, :, None] + keep, total)
    after = length + (~done).to(torch.int32)
    rank = (total / _penalty(after, s["alpha"])[:, :, None]).view(B, W * V)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :W]
    parent, token = order // V, order % V
    return {"parent": parent.to(torch.int32), "token": token.to(torch.int32), "new_score": total.view(B, W * V).gather(1, order).float(),
            "new_length": after.gather(1, parent), "new_finished": (done.gather(1, parent) | (token == s["eos"])).to(torch.int32)}


def _reorder(s):
    B, W, bs = s["B"], s["W"], s["bs"]
    parent, table, length = s["parent"].long(), s["table"].view(B, W, -1), s["kv_len"].long()
    n = table.shape[2]
    page, rem = length // bs, length % bs
    writing = table.gather(2, page[:, None, None].expand(B, W, 1))[:, :, 0].long()
    same = parent[:, :, None] == parent[:, None, :]
    first = ~(same & torch.ones((W, W), dtype=torch.bool, device="cuda").tril(-1)).any(dim=2)
    dead = ~(parent[:, None, :] == torch.arange(W, device="cuda")[None, :, None]).any(dim=2)
    free = torch.sort((~dead).to(torch.int8), dim=1, stable=True).indices          # the childless beams first
    spare = writing.gather(1, free)
    nth = (~first).cumsum(dim=1) - 1
    kept = writing.gather(1, parent)
    mine = torch.where(first, kept, spare.gather(1, nth.clamp(min=0)))
    at = torch.arange(n, device="cuda")[None, None, :]
    new = torch.where(at < page[:, None, None], table.gather(1, parent[:, :, None].expand(B, W, n)), table)
    new = torch.where(at == page[:, None, None], mine[:, :, None].to(new.dtype), new)
    b, w = torch.nonzero(~first & (rem > 0)[:, None], as_tuple=True)
    to, fr = mine[b, w], kept[b, w]
    rows = (torch.arange(bs, device="cuda")[None, :] < rem[b][:, None])[None, :, None, :, None]
    for k in ("k", "v"):
        bits = s[k].view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[s[k].element_size()])
        bits[:, to] = torch.where(rows, bits[:, fr], bits[:, to])
        if s[k + "s"] is not None:
            s[k + "s"][:, to] = s[k + "s"][:, fr]
    s["table"].copy_(new.view(B * W, n))
    return {k: s[k] for k in ("k", "v", "ks", "vs", "table") if s[k] is not None}


# --------------------------------------------------------------------------------- exact values
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("shared", "window"):
        return _exact_attention(case, s)
    if case["op"] == "select":
        B, W, V = case["B"], case["W"], case["V"]
        out = torch.empty((B, W), dtype=torch.float64, device="cuda")
        length, done = s["length"].tolist(), s["finished"].tolist()
        for b in range(B):
            rank, total = [], []
            for w in range(W):
                base = s["score"][b, w].double()
                if done[b][w]:
                    t = base[None]
                else:
                    t = base + torch.log_softmax(s["rows"][b * W + w, :V].double() / case["tau"], dim=0).topk(min(W, V)).values
                total.append(t)
                rank.append(t / ((5 + length[b][w] + (0 if done[b][w] else 1)) / 6) ** case["alpha"])
            rank, total = torch.cat(rank), torch.cat(total)
            out[b] = total[rank.topk(W).indices] if rank.numel() >= W else math.nan
        return {"parent": None, "token": None, "new_score": out, "new_length": None, "new_finished": None}
    # bits only move: the caches in 64 bits, page by page
    res = {}
    table, lens = s["table"].tolist(), s["kv_len"].tolist()
    for k in ("k", "v"):
        vals, scale = s[k].double(), None if s[k + "s"] is None else s[k + "s"].double()
        for b in range(case["B"]):
            page, rem = divmod(lens[b], case["bs"])
            par = s["parent"][b].tolist()
            pages = [table[b * case["W"] + w][page] for w in range(case["W"])]
            unused = [pages[w] for w in range(case["W"]) if w not in par]
            met = set()
            for p in par:
                if p in met:
                    to = unused.pop(0)
                    if rem:
                        vals[:, to, :, :rem] = vals[:, pages[p], :, :rem]
                        if scale is not None:
                            scale[:, to] = scale[:, pages[p]]
                met.add(p)
        res[k] = vals
        if scale is not None:
            res[k + "s"] = scale
    return {**{k: res[k] for k in ("k", "v", "ks", "vs") if k in res}, "table": None}


def _exact_attention(case, s):
    prefix, new = _lengths(case)
    table, bs, D = s["table"].cpu().tolist(), case["bs"], case["D"]
    G, out, lse, at = case["Hq"] // case["Hkv"], [], [], 0
    for r, (P, T) in enumerate(zip(prefix, new)):
        S = P + T
        bits = s["mask"][at:at + T]
        vis = torch.ones((T, S), dtype=torch.bool, device="cuda")
        for a in range(T):
            vis[:, P + a] = ((bits[:, a // 32] >> (a % 32)) & 1).bool()
        slots = torch.arange(S, device="cuda")
        if case["op"] == "window":
            depth = vis[:, P:].sum(dim=1) - 1
            pos = torch.cat([slots[:P], P + depth])
            vis &= (pos[None, :] > (P + depth)[:, None] - case["window"]) | (pos < case["sinks"])[None, :]
            slots = slots[vis.any(dim=0)]
            vis = vis[:, slots]
        ids = torch.tensor(table[r], device="cuda")[slots // bs]
        row = slots % bs
        o = torch.empty((T, case["Hq"], D), dtype=torch.float64, device="cuda")
        z = torch.empty((T, case["Hq"]), dtype=torch.float64, device="cuda")
        for h in range(case["Hkv"]):
            k, v = s["k"][ids, h, row].double(), s["v"][ids, h, row].double()
            x = (s["q"][at:at + T, h * G:(h + 1) * G].double().reshape(T * G, D) @ k.T) / math.sqrt(D)
            x = x.view(T, G, -1).masked_fill(~vis[:, None, :], -math.inf).view(T * G, -1)
            z[:, h * G:(h + 1) * G] = torch.logsumexp(x, dim=1).view(T, G)
            o[:, h * G:(h + 1) * G] = (torch.softmax(x, dim=1) @ v).view(T, G, D)
        out.append(o)
        lse.append(z)
        at += T
    return {"o": torch.cat(out), "lse": torch.cat(lse)}
