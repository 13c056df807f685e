"""Cases of the paged key/value cache and of the attention that decodes over it.

Five operators, each in its plain form (elementary torch operations) and, where ``own`` is true, as a
user calls it:

  sparse   fib_attn_tree_decode        a layer's window and rungs for a tree of drafted tokens over the cache
  dense    fib_attn_dense_tree_decode  the dense control for the same tree over the same cache
  commit   fib_attn_cache_commit       the accepted tokens of every layer into the cache's pages
  fork     fib_attn_cache_fork         sequences that take over, share or give back pages
  compact  fib_attn_cache_compact      the pages in use moved to the lowest ids

The cache holds, for every layer, pages of ``P`` rows: K rotated at its own position and V, both in the
type of the inputs, as pools [layers, pages, heads, P, 64]; ``table`` [sequences, entries] names the page
of rows jP .. jP+P-1 of a sequence, ``lens`` its rows, ``refs`` how many sequences hold a page.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
D = 64
FIB = [1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 610, 987]


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one sequence at the training length: a decode step of a single stream
        {"name": "sparse-token-1024", "op": "sparse", "dtype": "bf16", "B": 1, "Hq": 8, "H": 8, "T": 1, "depth": 0,
         "len": 1023, "P": 64, "W": 12, "mode": "mask", "base": "fib", "alpha": 1.5, "ragged": False},
        # odd heads in float32, learned alpha: seven drafts, two query heads to a key head
        {"name": "sparse-tree-f32-gqa", "op": "sparse", "dtype": "f32", "B": 5, "Hq": 6, "H": 3, "T": 7, "depth": 3,
         "len": 4095, "P": 16, "W": 10, "mode": "interp", "base": "fib", "alpha": 1.0371, "ragged": True},
        # a full batch whose drafts are checked at once: 64 sequences, trees of 64 nodes, lengths up to 16384
        {"name": "sparse-tree-b64", "op": "sparse", "dtype": "bf16", "B": 64, "Hq": 8, "H": 8, "T": 64, "depth": 7,
         "len": 16384, "P": 64, "W": 12, "mode": "interp", "base": "fib", "alpha": 0.9712, "ragged": False},
        # one new token of one sequence, dense control
        {"name": "dense-token-4096", "op": "dense", "dtype": "bf16", "B": 1, "Hq": 8, "H": 8, "T": 1, "depth": 0,
         "len": 4095, "P": 64, "ragged": False},
        # float32, shared key heads, five drafts, ragged short contexts
        {"name": "dense-tree-f32-gqa", "op": "dense", "dtype": "f32", "B": 6, "Hq": 8, "H": 4, "T": 5, "depth": 2,
         "len": 8191, "P": 32, "ragged": True},
        # a batch of long contexts with trees of 24 nodes: the cache is read from memory once
        {"name": "dense-tree-65536", "op": "dense", "dtype": "bf16", "B": 16, "Hq": 8, "H": 8, "T": 24, "depth": 5,
         "len": 65536, "P": 64, "ragged": False},
        # every sequence of a batch gains the one token that a decode step made, in all 16 layers
        {"name": "commit-token-b32", "op": "commit", "dtype": "bf16", "B": 32, "L": 16, "H": 8, "P": 16, "T": 1,
         "len": 260, "group": 1, "path": False},
        # beams in groups of eight that share their prompt's pages accept up to eight of 16 drafts: their last
        # page, partly filled, is copied before it is written
        {"name": "commit-beams-b64", "op": "commit", "dtype": "bf16", "B": 64, "L": 16, "H": 8, "P": 64, "T": 16,
         "len": 1000, "group": 8, "path": True},
        # beams of one step reordered: some double, some end
        {"name": "fork-beams-32", "op": "fork", "B": 32, "P": 64, "len": 4096, "spare": 100},
        # a large pool of small pages, 256 sequences
        {"name": "fork-slots-256", "op": "fork", "B": 256, "P": 16, "len": 8192, "spare": 5000},
        # a small pool after a few sequences have ended
        {"name": "compact-small", "op": "compact", "dtype": "f32", "L": 2, "H": 8, "P": 16, "pages": 300, "B": 7},
        # 2 GB of pages of the 16 layers, every second one free
        {"name": "compact-16-layers", "op": "compact", "dtype": "bf16", "L": 16, "H": 8, "P": 64, "pages": 1024, "B": 24},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sparse", "sparse", "dense", "dense", "commit", "commit", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("sparse", "dense"):
        H = rng.choice([1, 2, 3, 4, 8])
        G = rng.choice([1, 1, 1, 2, 3, 4])
        T = _log(rng, 1, 64)
        c = {"op": op, "dtype": dtype, "Hq": H * G, "H": H, "T": T, "depth": rng.randint(0, T - 1),
             "P": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.5}
        if op == "sparse":
            c["B"] = _log(rng, 1, 64)
            c["len"] = _log(rng, 1, 16384)
            c.update(W=rng.choice([1, 8, 10, 12, 24]), mode=rng.choice(["mask", "interp"]),
                     base=rng.choice(["fib", "pow2"]), alpha=round(rng.uniform(0.5, 1.5), 4))
        else:
            c["B"] = _log(rng, 1, 32)
            # no more than a quarter of the largest listed case's products
            most = 16 * 65536 * 8 * 24 // (4 if dtype == "bf16" else 16)
            c["len"] = _log(rng, 1, max(2, min(65536, most // (c["B"] * c["Hq"] * T))))
        return c
    if op == "commit":
        prompt = rng.random() < 0.3  # a prompt of up to 2048 tokens, or a few drafts
        T = _log(rng, 16, 2048) if prompt else _log(rng, 1, 64)
        B = _log(rng, 1, 4 if prompt else 64)
        return {"op": op, "dtype": dtype, "B": B, "L": rng.choice([1, 2, 6, 16]), "H": rng.choice([1, 3, 8]),
                "P": rng.choice([16, 32, 64, 128]), "T": T, "len": _log(rng, 1, 1000),
                "group": 1 if prompt else rng.choice([1, 2, 4]), "path": (not prompt) and rng.random() < 0.6}
    if op == "fork":
        return {"op": op, "B": _log(rng, 1, 256), "P": rng.choice([16, 32, 64, 128]), "len": _log(rng, 1, 8192),
                "spare": _log(rng, 1, 20000)}
    return {"op": op, "dtype": dtype, "L": rng.choice([1, 2, 4, 16]), "H": rng.choice([1, 3, 8]),
            "P": rng.choice([16, 32, 64]), "pages": _log(rng, 8, 500), "B": _log(rng, 1, 32)}


# ------------------------------------------------------------------------------------------ inputs
def _lens(B, most):
    """Lengths from short to `most`: an empty sequence and one of a single row among four or more."""
    v = [max(0, most * (i + 1) // B - (i * 13) % 29) for i in range(B)]
    v[-1] = most
    if B >= 4:
        v[0], v[1] = 0, 1
    return v


def _n_nodes(B, T, ragged):
    v = [T - (i % 4) * T // 4 if ragged else T for i in range(B)]
    if ragged and B >= 4:
        v[0] = 0
    return v


def _depths(T, depth):
    """Depths of the nodes: a spine 0..depth, then more branches of every depth."""
    return [s if s <= depth else (s - depth - 1) % (depth + 1) for s in range(T)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _rand_pool(shape, dtype, g):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _distances(case, N):
    """[(lo, w)] of the layer's rungs: mask mode the distinct rounded distances, interp mode the two
    bracketing rows' distance and the second one's weight."""
    base = FIB if case["base"] == "fib" else [1 << k for k in range(20) if (1 << k) < N]
    W = case["W"]
    if case["mode"] == "mask":
        d = sorted({round(case["alpha"] * f) for f in base})  # half to even
        return [(x, 0.0) for x in d if W <= x <= N - 1]
    a = float(np.float32(case["alpha"]))  # a learned alpha is held in float32
    return [(int(math.floor(a * f)), a * f - math.floor(a * f)) for f in base if W - 1 < a * f <= N - 1]


def _sequence_length(case):
    return case["len"] + case["T"]


def _prepare_attention(case, seed):
    B, Hq, H, T, P = case["B"], case["Hq"], case["H"], case["T"], case["P"]
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    lens = np.asarray(_lens(B, case["len"]))[r.permutation(B)]
    nodes = np.asarray(_n_nodes(B, T, case["ragged"]))[r.permutation(B)]
    depth = _depths(T, case["depth"])
    at = {}
    parent = np.full((B, T), -1, np.int64)
    for s in range(T):
        if depth[s]:
            parent[:, s] = np.asarray(at[depth[s] - 1])[r.randint(0, len(at[depth[s] - 1]), B)]
        at.setdefault(depth[s], []).append(s)
    MP = -(-case["len"] // P)
    used = [-(-int(n) // P) for n in lens]
    NP = sum(used) + 3
    ids = r.permutation(NP)
    table = np.full((B, MP), -1, np.int64)
    refs = np.zeros(NP, np.int64)
    first = 0
    for b in range(B):
        table[b, :used[b]] = ids[first:first + used[b]]
        first += used[b]
    refs[ids[:first]] = 1
    s = {"case": case, "q": _randn((B, Hq, T, D), dt, g), "k_new": _randn((B, H, T, D), dt, g),
         "v_new": _randn((B, H, T, D), dt, g), "k": _rand_pool((1, NP, H, P, D), dt, g),
         "v": _rand_pool((1, NP, H, P, D), dt, g), "table": _i32(table), "lens": _i32(lens), "refs": _i32(refs),
         "parent": _i32(parent), "nodes": _i32(nodes), "N": _sequence_length(case),
         "o": torch.zeros((B, Hq, T, D), device="cuda", dtype=dt),
         "lse": torch.zeros((B, Hq, T), device="cuda", dtype=torch.float32)}
    if case["op"] == "sparse":
        d = _distances(case, s["N"])
        s["lo"] = torch.tensor(list(range(case["W"])) + [x for x, _ in d], device="cuda", dtype=torch.int64)
        s["w"] = torch.tensor([0.0] * case["W"] + [w for _, w in d], device="cuda", dtype=torch.float64)
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        W, mode, base = case.get("W", 1), case.get("mode", "mask"), case.get("base", "fib")
        s["plan"] = fa.fib_attn_plan_create(
            fa.FIB_BASE_FIBONACCI if base == "fib" else fa.FIB_BASE_POW2, [case.get("alpha", 1.0)], W, s["N"],
            fa.FIB_MODE_MASK if mode == "mask" else fa.FIB_MODE_INTERP)
        s["alpha"] = torch.tensor([case["alpha"]], device="cuda", dtype=torch.float32) if mode == "interp" else None
        s["cache"] = _own_cache(fa, s, dt)
        if case["op"] == "dense":
            need = fa.fib_attn_dense_tree_workspace_size(s["plan"], s["cache"], B, Hq, T)
            s["workspace"] = torch.empty(max(need, 1), device="cuda", dtype=torch.uint8)
    return s


def _own_cache(fa, s, dt):
    L, NP, H, P = s["k"].shape[:4]
    cache = fa.fib_attn_cache_create(L, H, P, NP, s["table"].shape[0], s["table"].shape[1], dt, k=s["k"], v=s["v"])
    cache.table.copy_(s["table"])
    cache.lens.copy_(s["lens"])
    cache.refs.copy_(s["refs"])
    return cache


def _prepare_commit(case, seed):
    B, L, H, P, T, G = (case[x] for x in ("B", "L", "H", "P", "T", "group"))
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    n_new = np.asarray([1 + (i * 5) % max(1, -(-T // 2)) if case["path"] else T - (i % 3) * T // 8 for i in range(B)])
    if B >= 4:
        n_new[1] = 0  # a slot that takes no part
    n_new = n_new[r.permutation(B)]
    groups = -(-B // G)
    lens_g = [max(0, case["len"] - (i * 7) % (P + 1)) for i in range(groups)]
    lens = np.asarray([lens_g[b // G] for b in range(B)])
    MP = -(-(case["len"] + T) // P)
    held = [-(-n // P) for n in lens_g]
    NP = sum(held) + B * (2 + -(-T // P))
    ids = r.permutation(NP)
    table = np.full((B, MP), -1, np.int64)
    refs = np.zeros(NP, np.int64)
    first = 0
    for i in range(groups):
        pages = ids[first:first + held[i]]
        first += held[i]
        for b in range(i * G, min(B, (i + 1) * G)):
            table[b, :held[i]] = pages
            refs[pages] += 1
    path = np.tile(np.arange(T), (B, 1))
    if case["path"]:  # slots of a root-to-node path, ascending
        for b in range(B):
            path[b, :n_new[b]] = np.sort(r.choice(T, n_new[b], replace=False))
    s = {"case": case, "k_new": _randn((L, B, H, T, D), dt, g), "v_new": _randn((L, B, H, T, D), dt, g),
         "k": _rand_pool((L, NP, H, P, D), dt, g), "v": _rand_pool((L, NP, H, P, D), dt, g), "table": _i32(table),
         "lens": _i32(lens), "refs": _i32(refs), "n_new": _i32(n_new), "path": _i32(path)}
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        s["plan"] = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.0] * L, 12, case["len"] + T, fa.FIB_MODE_MASK)
        _own_state(fa, s, dt)
    return s


def _own_state(fa, s, dt):
    """The cache, its tables as they stand before a pass, and the scratch."""
    s["cache"] = _own_cache(fa, s, dt)
    s["before"] = s["cache"].meta.clone()
    s["workspace"] = torch.empty(max(1, fa.fib_attn_cache_workspace_size(s["cache"])), device="cuda", dtype=torch.uint8)


def _prepare_fork(case, seed):
    B, P = case["B"], case["P"]
    r = np.random.RandomState(seed % (1 << 31))
    lens = np.asarray(_lens(B, case["len"]))[r.permutation(B)]
    MP = -(-case["len"] // P)
    used = [-(-int(n) // P) for n in lens]
    NP = sum(used) + case["spare"]
    ids = r.permutation(NP)
    table = np.full((B, MP), -1, np.int64)
    first = 0
    for b in range(B):
        table[b, :used[b]] = ids[first:first + used[b]]
        first += used[b]
    refs = np.zeros(NP, np.int64)
    refs[ids[:first]] = 1
    src = r.randint(-1, B, B)  # any sequence may go on in any slot; -1 ends one
    src = np.where(r.rand(B) < 0.3, np.arange(B), src)
    s = {"case": case, "table": _i32(table), "lens": _i32(lens), "refs": _i32(refs), "src": _i32(src)}
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        s["k"] = torch.empty((1, NP, 1, P, D), device="cuda", dtype=torch.bfloat16)
        s["v"] = torch.empty((1, NP, 1, P, D), device="cuda", dtype=torch.bfloat16)
        _own_state(fa, s, torch.bfloat16)
    return s


def _prepare_compact(case, seed):
    B, L, H, P, NP = (case[x] for x in ("B", "L", "H", "P", "pages"))
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    each = max(1, NP // (2 * B))
    live = min(NP, each * B)
    MP = -(-NP // B) + 1
    ids = r.permutation(NP)
    table = np.full((B, MP), -1, np.int64)
    refs = np.zeros(NP, np.int64)
    lens = np.zeros(B, np.int64)
    for b in range(B):
        pages = ids[b * each:(b + 1) * each][:max(0, live - b * each)]
        table[b, :len(pages)] = pages
        refs[pages] += 1
        lens[b] = max(0, len(pages) * P - r.randint(0, P))
    if B >= 2:  # two sequences that share a prompt
        n = int((table[0] >= 0).sum()) // 2
        old = table[1, :n][table[1, :n] >= 0]
        refs[old] -= 1
        table[1, :n] = np.where(table[1, :n] >= 0, table[0, :n], -1)
        refs[table[1, :n][table[1, :n] >= 0]] += 1
    s = {"case": case, "k": _rand_pool((L, NP, H, P, D), dt, g), "v": _rand_pool((L, NP, H, P, D), dt, g),
         "table": _i32(table), "lens": _i32(lens), "refs": _i32(refs)}
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        _own_state(fa, s, dt)
    return s


def prepare(case, seed):
    op = case["op"]
    if op in ("sparse", "dense"):
        return _prepare_attention(case, seed)
    return {"commit": _prepare_commit, "fork": _prepare_fork, "compact": _prepare_compact}[op](case, seed)


# ------------------------------------------------------------------------------------------ plain forms
def _rope(x, pos):
    """Rotate-half pairs (m, m + 32) of x by pos * 10000^(-m/32), the angle in 64 bits."""
    m = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(10000.0, device=x.device, dtype=torch.float64), -m / 32)
    c, s = torch.cos(a).float(), torch.sin(a).float()
    x1, x2 = x[..., :D // 2].float(), x[..., D // 2:].float()
    return torch.cat([x1 * c - x2 * s, x1 * s + x2 * c], dim=-1)


def _ancestors(parent):
    """anc[b, s, u]: u is s or above it; depth[b, s]."""
    T = parent.shape[1]
    u = torch.arange(T, device=parent.device)
    step = ((parent[:, :, None] == u) | (u[:, None] == u)).float()
    step = (step @ step > 0).float()  # paths of at most 2, 4, ... 64 steps
    step = (step @ step > 0).float()
    step = (step @ step > 0).float()
    step = (step @ step > 0).float()
    step = (step @ step > 0).float()
    step = (step @ step > 0).float()
    return step > 0, step.sum(-1).long() - 1


def _plain_sparse(s):
    c = s["case"]
    B, Hq, H, T, P = c["B"], c["Hq"], c["H"], c["T"], c["P"]
    G = Hq // H
    dev = s["q"].device
    anc, depth = _ancestors(s["parent"].long())
    pos = s["lens"].long()[:, None] + depth  # [B, T]
    q = _rope(s["q"], pos[:, None, :])
    kd, vd = _rope(s["k_new"], pos[:, None, :]), s["v_new"].float()
    table = s["table"].long().clamp(min=0)
    bi = torch.arange(B, device=dev)[:, None, None]

    def rows(dist):  # K and V [B, H, T, keys, 64] of the tokens `dist` before each node
        back = depth[:, :, None] - dist
        hit = anc[:, :, None, :] & (depth[:, None, None, :] == back[..., None])
        at = hit.float().argmax(-1)  # the ancestor at that depth
        row = (pos[:, :, None] - dist).clamp(min=0)
        row = torch.minimum(row, (s["lens"].long()[:, None, None] - 1).clamp(min=0))
        page = table[bi, (row // P).clamp(max=table.shape[1] - 1)]
        new = (back >= 0)[:, None, :, :, None]
        out = []
        for pool, fresh in ((s["k"], kd), (s["v"], vd)):
            old = pool[0][page, :, row % P].permute(0, 3, 1, 2, 4).float()
            now = fresh[bi, :, at].permute(0, 3, 1, 2, 4)
            out.append(torch.where(new, now, old))
        return out

    lo, w = s["lo"], s["w"].float()
    k, v = rows(lo)
    if c["mode"] == "interp":
        k1, v1 = rows(lo + 1)
        k = torch.where(w[:, None] > 0, (1 - w)[:, None] * k + w[:, None] * k1, k)
        v = torch.where(w[:, None] > 0, (1 - w)[:, None] * v + w[:, None] * v1, v)
    need = lo + (s["w"] > 0)
    ok = need <= pos[:, :, None]
    qg = q.view(B, H, G, T, D)
    sc = (qg[:, :, :, :, None, :] * k[:, :, None]).sum(-1) / 8
    sc = torch.where(ok[:, None, None], sc, torch.tensor(-math.inf, device=dev))
    mx = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - mx)
    z = p.sum(-1, keepdim=True)
    o = ((p / z)[..., None] * v[:, :, None]).sum(-2).view(B, Hq, T, D)
    lse = (mx + torch.log(z))[..., 0].view(B, Hq, T)
    on = (torch.arange(T, device=dev) < s["nodes"][:, None])[:, None]
    return [torch.where(on[..., None], o, torch.tensor(0.0, device=dev)).to(s["q"].dtype),
            torch.where(on, lse, torch.tensor(0.0, device=dev))]


def _plain_dense(s):
    c = s["case"]
    B, Hq, H, T, P = c["B"], c["Hq"], c["H"], c["T"], c["P"]
    dev = s["q"].device
    anc, depth = _ancestors(s["parent"].long())
    lens = s["lens"].long()
    pos = lens[:, None] + depth
    q = _rope(s["q"], pos[:, None, :]).view(B, H, -1, D)  # the G query heads of a key head after one another
    kd, vd = _rope(s["k_new"], pos[:, None, :]), s["v_new"].float()
    table = s["table"].long().clamp(min=0)
    MP = table.shape[1]
    k = s["k"][0][table].permute(0, 2, 1, 3, 4).reshape(B, H, MP * P, D).float()
    v = s["v"][0][table].permute(0, 2, 1, 3, 4).reshape(B, H, MP * P, D).float()
    inf = torch.tensor(-math.inf, device=dev)
    live = torch.arange(MP * P, device=dev) < lens[:, None]
    old = torch.where(live[:, None, None], q @ k.transpose(-1, -2) / 8, inf)
    new = (q @ kd.transpose(-1, -2) / 8).view(B, H, -1, T, T)
    new = torch.where(anc[:, None, None], new, inf).view(B, H, -1, T)
    mx = torch.maximum(old.amax(-1, keepdim=True), new.amax(-1, keepdim=True))
    old, new = torch.exp(old - mx), torch.exp(new - mx)
    z = old.sum(-1, keepdim=True) + new.sum(-1, keepdim=True)
    o = ((old @ v + new @ vd) / z).view(B, Hq, T, D)
    lse = (mx + torch.log(z)).view(B, Hq, T)
    on = (torch.arange(T, device=dev) < s["nodes"][:, None])[:, None]
    zero = torch.tensor(0.0, device=dev)
    return [torch.where(on[..., None], o, zero).to(s["q"].dtype), torch.where(on, lse, zero)]


def _plain_commit(s):
    c = s["case"]
    B, P, T = c["B"], c["P"], c["T"]
    dev = s["k"].device
    lens, n, refs = s["lens"].long(), s["n_new"].long(), s["refs"].long()
    table = s["table"].long()
    MP = table.shape[1]
    b = torch.arange(B, device=dev)
    part = (lens % P != 0) & (n > 0)
    at = (lens // P).clamp(max=MP - 1)
    page = torch.where(part, table[b, at], -1)
    same = (page[:, None] == page) & part[:, None] & part
    last = ~(same & (b[None, :] > b[:, None])).any(1)
    count = refs[page.clamp(min=0)]
    keep = (count <= 1) | (last & (same.sum(1) == count))
    copy = part & ~keep
    first = (lens + P - 1) // P
    end = torch.where(n > 0, (lens + n + P - 1) // P, first)
    need = copy.long() + end - first
    off = need.cumsum(0) - need
    free = (refs == 0).nonzero().flatten()
    j = torch.arange(MP, device=dev)
    fresh = (j >= first[:, None]) & (j < end[:, None])
    slot = (off + copy.long())[:, None] + j - first[:, None]
    table = torch.where(fresh, free[torch.where(fresh, slot, 0)], table)
    dst = free[torch.where(copy, off, 0)]
    table[b[copy], at[copy]] = dst[copy]
    refs = refs.index_add(0, page[copy], -torch.ones_like(page[copy]))
    refs[free[:int(need.sum())]] = 1
    # the rows of a shared last page, then the new rows
    r = torch.arange(P, device=dev)
    cb, cr = (copy[:, None] & (r < (lens % P)[:, None])).nonzero(as_tuple=True)
    nb, ni = (torch.arange(T, device=dev) < n[:, None]).nonzero(as_tuple=True)
    pos = lens[nb] + ni
    node = s["path"].long()[nb, ni]
    to = table[nb, pos // P]
    k, v = s["k"], s["v"]
    k[:, dst[cb], :, cr] = k[:, page[cb], :, cr]
    v[:, dst[cb], :, cr] = v[:, page[cb], :, cr]
    k[:, to, :, pos % P] = _rope(s["k_new"][:, nb, :, node], pos[:, None, None]).to(k.dtype)
    v[:, to, :, pos % P] = s["v_new"][:, nb, :, node]
    return [k, v, table.int(), (lens + n).int(), refs.int()]


def _plain_fork(s):
    P = s["case"]["P"]
    dev = s["table"].device
    lens, src, refs, table = s["lens"].long(), s["src"].long(), s["refs"].long(), s["table"].long()
    j = torch.arange(table.shape[1], device=dev)
    held = j < ((lens + P - 1) // P)[:, None]
    gone = src < 0
    at = src.clamp(min=0)
    now = torch.where(gone, 0, lens[at])
    keeps = j < ((now + P - 1) // P)[:, None]
    out = torch.where(keeps, table[at], -1)
    out = torch.where(keeps | held, out, table)  # entries behind both lengths stay
    one = torch.ones((), device=dev, dtype=torch.int64)
    refs = refs.index_add(0, out[keeps], one.expand(int(keeps.sum())))
    refs = refs.index_add(0, table[held], -one.expand(int(held.sum())))
    return [out.int(), now.int(), refs.int()]


def _plain_compact(s):
    P = s["case"]["P"]
    refs, table = s["refs"].long(), s["table"].long()
    NP = refs.numel()
    live = refs > 0
    n = int(live.sum())
    ids = torch.arange(NP, device=refs.device)
    src = ids[live & (ids >= n)]
    dst = ids[~live & (ids < n)]
    remap = torch.where(live, ids, -1)
    remap[src] = dst
    k, v = s["k"], s["v"]
    k[:, dst] = k[:, src]
    v[:, dst] = v[:, src]
    j = torch.arange(table.shape[1], device=refs.device)
    held = j < ((s["lens"].long() + P - 1) // P)[:, None]
    table = torch.where(held, remap[table.clamp(min=0)], table)
    out = refs.clone()
    out[dst] = refs[src]
    out[src] = 0
    return [k, v, table.int(), out.int(), remap.int()]


def _run_own(s):
    from fibonacci_offset_sparse_gb300 import fib_attn as fa
    op = s["case"]["op"]
    if op == "sparse":
        o, lse = fa.fib_attn_tree_decode(s["plan"], 0, s["cache"], s["q"], s["k_new"], s["v_new"], parent=s["parent"],
                                         n_nodes=s["nodes"], o=s["o"], lse=s["lse"], alpha_dev=s["alpha"])
        return [o, lse]
    if op == "dense":
        o, lse = fa.fib_attn_dense_tree_decode(s["plan"], 0, s["cache"], s["q"], s["k_new"], s["v_new"],
                                               parent=s["parent"], n_nodes=s["nodes"], o=s["o"], lse=s["lse"],
                                               workspace=s["workspace"])
        return [o, lse]
    cache = s["cache"]
    cache.meta.copy_(s["before"])  # back to the tables as they stood: a pass starts where the last one did
    if op == "commit":
        fa.fib_attn_cache_commit(s["plan"], cache, s["k_new"], s["v_new"], s["n_new"],
                                 path=s["path"] if s["case"]["path"] else None, workspace=s["workspace"])
        return [cache.k, cache.v, cache.table, cache.lens, cache.refs]
    if op == "fork":
        fa.fib_attn_cache_fork(cache, s["src"], workspace=s["workspace"])
        return [cache.table, cache.lens, cache.refs]
    remap = fa.fib_attn_cache_compact(cache, workspace=s["workspace"])
    return [cache.k, cache.v, cache.table, cache.refs, remap]


def run(state):
    if own:
        return _run_own(state)
    return {"sparse": _plain_sparse, "dense": _plain_dense, "commit": _plain_commit, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op = case["op"]
    es = 2 if case.get("dtype") == "bf16" else 4
    row = D * es
    if op in ("sparse", "dense"):
        B, Hq, H, T = case["B"], case["Hq"], case["H"], case["T"]
        lens, nodes = _lens(B, case["len"]), _n_nodes(B, T, case["ragged"])
        n = sum(nodes)
        io = n * Hq * (2 * row + 4) + n * H * 2 * row + B * 8 + n * 4
        if op == "dense":
            # which sequence has which number of nodes goes by the seed: the mean
            keys = sum(lens)
            return {"bytes": io + keys * H * 2 * row, "flops": keys * (n / B) * Hq * 4 * D + n * Hq * (case["depth"] + 1) * 4 * D}
        rungs = _distances(case, _sequence_length(case))
        two = 1 if case["mode"] == "interp" else 0
        levels = min(case["depth"], T - 1) + 1
        rows = sum(min(x, case["W"] - 1 + len(rungs) * (levels + two)) for x in lens)
        keys = sum(1 for _ in rungs) * (1 + two) + case["W"]
        return {"bytes": io + rows * H * 2 * row, "flops": n * Hq * keys * 4 * D}
    if op == "commit":
        B, L, H, P, T, G = (case[x] for x in ("B", "L", "H", "P", "T", "group"))
        n = [1 + (i * 5) % max(1, -(-T // 2)) if case["path"] else T - (i % 3) * T // 8 for i in range(B)]
        if B >= 4:
            n[1] = 0
        copied = 0
        if G > 1:
            for i in range(-(-B // G)):
                copied += (min(G, B - i * G) - 1) * (max(0, case["len"] - (i * 7) % (P + 1)) % P)
        return {"bytes": (sum(n) + copied) * L * H * 4 * row + 8 * B, "flops": sum(n) * L * H * 6 * D / 2}
    if op == "fork":
        held = sum(-(-x // case["P"]) for x in _lens(case["B"], case["len"]))
        return {"bytes": 4 * (3 * held + 3 * case["B"]), "flops": 0}
    B, L, H, P, NP = (case[x] for x in ("B", "L", "H", "P", "pages"))
    live = min(NP, max(1, NP // (2 * B)) * B)
    moved = live * (NP - live) / NP  # of pages spread evenly over the pool
    return {"bytes": moved * L * H * P * 4 * row + 12 * NP, "flops": 0}


# ------------------------------------------------------------------------------------------ 64 bits
def _turned(x, pos):
    """x [..., 64] as 32 complex numbers turned by pos: back as 64 reals, in 64 bits."""
    x = x.double()
    z = torch.complex(x[..., :32], x[..., 32:])
    m = torch.arange(32, device=x.device, dtype=torch.float64)
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64).expand(pos.shape + (32,)),
                       pos.double()[..., None] * torch.exp(-m / 32 * math.log(10000.0)))
    z = z * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_attention(case, seed):
    s = prepare(case, seed)
    B, Hq, H, T, P = case["B"], case["Hq"], case["H"], case["T"], case["P"]
    G = Hq // H
    o = torch.zeros((B, Hq, T, D), device="cuda", dtype=torch.float64)
    lse = torch.zeros((B, Hq, T), device="cuda", dtype=torch.float64)
    lens, nodes, parent = s["lens"].tolist(), s["nodes"].tolist(), s["parent"].tolist()
    rungs = _distances(case, s["N"]) if case["op"] == "sparse" else None
    for b in range(B):
        n, length = nodes[b], lens[b]
        if not n:
            continue
        chain = []  # the slots from a node up to its root
        for u in range(n):
            chain.append([u] + (chain[parent[b][u]] if parent[b][u] >= 0 else []))
        depth = torch.tensor([len(x) - 1 for x in chain], device="cuda")
        pages = s["table"][b, :-(-length // P)].long()
        K = s["k"][0, pages].double().transpose(1, 2).reshape(-1, H, D)[:length]
        V = s["v"][0, pages].double().transpose(1, 2).reshape(-1, H, D)[:length]
        K = torch.cat([K, _turned(s["k_new"][b, :, :n], length + depth).transpose(0, 1)])
        V = torch.cat([V, s["v_new"][b, :, :n].double().transpose(0, 1)])
        q = _turned(s["q"][b, :, :n], length + depth).view(H, G, n, D)
        # weight[u, key]: node u's share of each row in each of its keys, dense or by distance
        if rungs is None:
            sees = torch.zeros((n, length + n), device="cuda", dtype=torch.bool)
            sees[:, :length] = True
            for u in range(n):
                sees[u, [length + a for a in chain[u]]] = True
            sc = torch.einsum("hgtd,khd->hgtk", q, K) / 8
            sc = sc.masked_fill(~sees, -math.inf)
            lse[b, :, :n] = torch.logsumexp(sc, -1).view(Hq, n)
            o[b, :, :n] = torch.einsum("hgtk,khd->hgtd", torch.softmax(sc, -1), V).reshape(Hq, n, D)
            continue
        keys = [(x, 0.0) for x in range(case["W"])] + rungs
        one, two, share, live = [], [], [], []
        for u in range(n):
            where = lambda d: length + chain[u][d] if d < len(chain[u]) else length + len(chain[u]) - 1 - d  # noqa: E731
            p = length + len(chain[u]) - 1
            on = [x + (w > 0) <= p for x, w in keys]
            one.append([where(x) if a else 0 for (x, w), a in zip(keys, on)])
            two.append([where(x + 1) if a and w > 0 else 0 for (x, w), a in zip(keys, on)])
            share.append([w for _, w in keys])
            live.append(on)
        one, two = torch.tensor(one, device="cuda"), torch.tensor(two, device="cuda")
        w = torch.tensor(share, device="cuda", dtype=torch.float64)[..., None, None]
        live = torch.tensor(live, device="cuda")
        k = (1 - w) * K[one] + w * torch.where(w > 0, K[two], 0.0)
        v = (1 - w) * V[one] + w * torch.where(w > 0, V[two], 0.0)
        sc = torch.einsum("hgtd,tkhd->hgtk", q, k) / 8
        sc = sc.masked_fill(~live, -math.inf)
        lse[b, :, :n] = torch.logsumexp(sc, -1).view(Hq, n)
        o[b, :, :n] = torch.einsum("hgtk,tkhd->hgtd", torch.softmax(sc, -1), v).reshape(Hq, n, D)
    return [o, lse]


def _exact_commit(case, seed):
    s = prepare(case, seed)
    P = case["P"]
    k, v = s["k"].double(), s["v"].double()
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    n_new, path = s["n_new"].tolist(), s["path"].tolist()
    wants = {}  # page -> the sequences that would write into it
    for b, n in enumerate(n_new):
        if n and lens[b] % P:
            wants.setdefault(table[b][lens[b] // P], []).append(b)
    free = iter([p for p, c in enumerate(refs) if not c])
    before = list(refs)
    for b, n in enumerate(n_new):
        if not n:
            continue
        if lens[b] % P:
            page = table[b][lens[b] // P]
            others = wants[page]
            if before[page] > 1 and not (len(others) == before[page] and b == others[-1]):
                to = next(free)
                rows = lens[b] % P
                k[:, to, :, :rows] = k[:, page, :, :rows]
                v[:, to, :, :rows] = v[:, page, :, :rows]
                refs[page] -= 1
                refs[to] = 1
                table[b][lens[b] // P] = to
        for j in range(-(-lens[b] // P), -(-(lens[b] + n) // P)):
            table[b][j] = next(free)
            refs[table[b][j]] = 1
    nb = torch.tensor([b for b, n in enumerate(n_new) for _ in range(n)], device="cuda", dtype=torch.int64)
    pos = [lens[b] + i for b, n in enumerate(n_new) for i in range(n)]
    node = torch.tensor([path[b][i] for b, n in enumerate(n_new) for i in range(n)], device="cuda", dtype=torch.int64)
    to = torch.tensor([table[b][p // P] for b, p in zip(nb.tolist(), pos)], device="cuda", dtype=torch.int64)
    pos = torch.tensor(pos, device="cuda", dtype=torch.int64)
    k[:, to, :, pos % P] = _turned(s["k_new"][:, nb, :, node], pos[:, None, None])
    v[:, to, :, pos % P] = s["v_new"][:, nb, :, node].double()
    return [k, v, np.asarray(table, np.int32), np.asarray([x + n for x, n in zip(lens, n_new)], np.int32),
            np.asarray(refs, np.int32)]


def _exact_fork(case, seed):
    s = prepare(case, seed)
    P = case["P"]
    table, lens, refs, src = (s[x].tolist() for x in ("table", "lens", "refs", "src"))
    new, now = [list(x) for x in table], []
    for b, a in enumerate(src):
        now.append(lens[a] if a >= 0 else 0)
        for j in range(-(-lens[b] // P)):
            refs[table[b][j]] -= 1
            new[b][j] = -1
        for j in range(-(-now[b] // P)):
            new[b][j] = table[a][j]
            refs[new[b][j]] += 1
    return [np.asarray(new, np.int32), np.asarray(now, np.int32), np.asarray(refs, np.int32)]


def _exact_compact(case, seed):
    s = prepare(case, seed)
    P = case["P"]
    table, lens, refs = (s[x].tolist() for x in ("table", "lens", "refs"))
    n = sum(c > 0 for c in refs)
    holes = iter([p for p in range(n) if not refs[p]])
    remap = [p if c else -1 for p, c in enumerate(refs)]
    k, v = s["k"].double(), s["v"].double()
    for p in range(n, len(refs)):
        if refs[p]:
            to = next(holes)
            k[:, to], v[:, to] = k[:, p], v[:, p]
            refs[to], refs[p], remap[p] = refs[p], 0, to
    for b, length in enumerate(lens):
        for j in range(-(-length // P)):
            table[b][j] = remap[table[b][j]]
    return [k, v, np.asarray(table, np.int32), np.asarray(refs, np.int32), np.asarray(remap, np.int32)]


def exact(case, seed):
    op = case["op"]
    if op in ("sparse", "dense"):
        return _exact_attention(case, seed)
    return {"commit": _exact_commit, "fork": _exact_fork, "compact": _exact_compact}[op](case, seed)
