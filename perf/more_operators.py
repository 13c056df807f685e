"""Cases of rotary positions by themselves and of eviction from the paged cache by accumulated attention weight.

Three operators, each in its plain form (elementary torch operations) and, where ``own`` is true, as a
user calls it:

  rotary  fib_attn_rotary        queries and keys turned by their positions, or gradients turned back
  weigh   fib_attn_cache_weigh   the attention weight that new tokens give to each cached row, added up
  evict   fib_attn_cache_evict   all but the first, the last and the heaviest rows leave the cache

The cache holds, for every layer, pages of ``P`` rows: K and V as pools [layers, pages, heads, P, 64]; ``table``
[sequences, entries] names the page of rows jP .. jP+P-1 of a sequence, ``lens`` its rows, ``refs`` how many
sequences hold a page.  ``weights`` [layers, sequences, heads, rows], float32, is what each row was given so far.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
D = 64
BASE = 10000.0


# ------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step of one stream: the new token's query and key heads, at the position that the cache's length says
        {"name": "rotary-token", "op": "rotary", "dtype": "bf16", "B": 1, "Hq": 8, "Hk": 8, "N": 1, "layout": "half", "R": 64,
         "scaling": "plain", "factor": 1.0, "pos": "start", "first": 1023, "fused": True, "back": False},
        # gradients of float32 queries and shared keys back into the projection's layout, half of the head, odd length
        {"name": "rotary-back-f32", "op": "rotary", "dtype": "f32", "B": 3, "Hq": 6, "Hk": 3, "N": 1023, "layout": "interleaved", "R": 32,
         "scaling": "linear", "factor": 4.0, "pos": "none", "first": 0, "fused": True, "back": True},
        # prompts at the evaluation length out of a fused projection [B, N, (8 + 8 + 8) * 64], stretched to four times the training length
        {"name": "rotary-prompt", "op": "rotary", "dtype": "bf16", "B": 8, "Hq": 8, "Hk": 8, "N": 4096, "layout": "half", "R": 64,
         "scaling": "yarn", "factor": 4.0, "pos": "none", "first": 0, "fused": True, "back": False},
        # one long row of packed documents, each with positions of its own; three quarters of the head
        {"name": "rotary-packed-131072", "op": "rotary", "dtype": "bf16", "B": 1, "Hq": 8, "Hk": 8, "N": 131072, "layout": "half", "R": 48,
         "scaling": "ntk", "factor": 8.0, "pos": "packed", "first": 0, "fused": False, "back": False},
        # drafts accepted by a few float32 sequences with two query heads to a key head
        {"name": "weigh-path-f32", "op": "weigh", "dtype": "f32", "L": 2, "B": 5, "Hq": 6, "H": 3, "T": 7, "len": 1000, "P": 16,
         "path": True, "set": False},
        # the token that every sequence of a batch has just gained, in all 16 layers
        {"name": "weigh-token-b32", "op": "weigh", "dtype": "bf16", "L": 16, "B": 32, "Hq": 8, "H": 8, "T": 1, "len": 2048, "P": 64,
         "path": False, "set": False},
        # the last 32 tokens of long prompts look back over them, before what they leave aside is evicted
        {"name": "weigh-window-8192", "op": "weigh", "dtype": "bf16", "L": 16, "B": 4, "Hq": 8, "H": 8, "T": 32, "len": 8192, "P": 64,
         "path": False, "set": True},
        # whole prompts, every token of them
        {"name": "weigh-prompt-2048", "op": "weigh", "dtype": "bf16", "L": 4, "B": 2, "Hq": 8, "H": 8, "T": 2048, "len": 2048, "P": 64,
         "path": False, "set": True},
        # a few short float32 sequences
        {"name": "evict-small-f32", "op": "evict", "dtype": "f32", "L": 2, "B": 3, "H": 3, "P": 16, "len": 200, "keep": 120, "sink": 4,
         "recent": 32, "group": 1},
        # beams in groups of four that share their prompt's pages
        {"name": "evict-beams", "op": "evict", "dtype": "bf16", "L": 16, "B": 16, "H": 8, "P": 32, "len": 2048, "keep": 1024, "sink": 4,
         "recent": 256, "group": 4},
        # a batch cut to half, all 16 layers
        {"name": "evict-b16-4096", "op": "evict", "dtype": "bf16", "L": 16, "B": 16, "H": 8, "P": 64, "len": 4096, "keep": 2048, "sink": 4,
         "recent": 512, "group": 1},
        # one long context cut to a quarter
        {"name": "evict-65536", "op": "evict", "dtype": "bf16", "L": 16, "B": 1, "H": 8, "P": 64, "len": 65536, "keep": 16384, "sink": 16,
         "recent": 2048, "group": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "weigh", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rotary":
        Hq = rng.choice([1, 2, 4, 8, 12])
        Hk = rng.choice([0, 1, Hq, max(1, Hq // 2)])
        B = _log(rng, 1, 64)
        N = _log(rng, 1, max(2, min(131072, 131072 * 16 // (B * (Hq + Hk) * (1 if dtype == "bf16" else 2)))))
        return {"op": op, "dtype": dtype, "B": B, "Hq": Hq, "Hk": Hk, "N": N, "layout": rng.choice(["half", "interleaved"]),
                "R": rng.choice([64, 64, 48, 32, 16, 20, 6, 2]), "scaling": rng.choice(["plain", "linear", "ntk", "yarn"]),
                "factor": round(rng.uniform(1.0, 16.0), 2), "pos": rng.choice(["none", "start", "packed"]), "first": _log(rng, 1, 60000),
                "fused": rng.random() < 0.5, "back": rng.random() < 0.4}
    H = rng.choice([1, 2, 3, 8])
    L = rng.choice([1, 2, 5, 16])
    P = rng.choice([16, 32, 64, 128])
    if op == "weigh":
        G = rng.choice([1, 1, 2, 3, 8])
        whole = rng.random() < 0.25  # a whole prompt, or what a step or a window of it gains
        T = _log(rng, 16, 2048) if whole else _log(rng, 1, 64)
        B = _log(rng, 1, 4 if whole else 32)
        rows = 16 * 4 * 8 * 8192 // (1 if dtype == "bf16" else 2)  # no more cached rows than the largest listed case ...
        most = min(16384, rows // (L * B * H))
        pairs = 16 * 4 * 8 * 8192 * 32 // 2  # ... and no more products
        most = max(2, min(most, pairs // (L * B * H * G * T) if not whole else T))
        while whole and L * B * H * G * T * T > pairs:
            T = max(1, T * 3 // 4)
        return {"op": op, "dtype": dtype, "L": L, "B": B, "Hq": H * G, "H": H, "T": T, "len": T if whole else max(T, _log(rng, 1, most)), "P": P,
                "path": (not whole) and rng.random() < 0.5, "set": whole or rng.random() < 0.3}
    B = _log(rng, 1, 32)
    length = _log(rng, 2, max(4, min(65536, 16 * 16 * 8 * 4096 // 2 // (L * B * H * (1 if dtype == "bf16" else 2)))))
    keep = max(1, min(length - 1, int(length * rng.uniform(0.1, 0.95))))
    sink = rng.randint(0, min(keep, 64) // 2)
    return {"op": op, "dtype": dtype, "L": L, "B": B, "H": H, "P": P, "len": length, "keep": keep, "sink": sink,
            "recent": rng.randint(0, (keep - sink) // 2), "group": rng.choice([1, 1, 2, 4])}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, dtype, g):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(generator=g)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device="cuda")


def _positions(case, r):
    """(explicit positions [B, N] or None, first positions [B] or None, one more than the last)."""
    B, N = case["B"], case["N"]
    if case["pos"] == "none":
        return None, None, N
    if case["pos"] == "start":
        first = case["first"] - (r.permutation(B) * 7) % (case["first"] + 1)
        return None, first, int(first.max()) + N
    # documents of some 900 tokens in a row, another cut in each row
    cut = r.rand(B, N) < 1.0 / 900
    cut[:, 0] = True
    at = np.arange(N)[None]
    pos = at - np.maximum.accumulate(np.where(cut, at, 0), axis=1)
    return pos, None, int(pos.max()) + 1


def _views(case, Hq, Hk, dt, g):
    """Queries and keys [B, H, N, 64]: views of a projection [B, N, heads * 64] (as many values follow as there are keys), or contiguous."""
    B, N = case["B"], case["N"]
    if case["fused"]:
        x = _randn((B, N, Hq + 2 * Hk, D), dt, g)
        return x, x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2) if Hk else None
    return None, _randn((B, Hq, N, D), dt, g), _randn((B, Hk, N, D), dt, g) if Hk else None


def _prepare_rotary(case, seed):
    B, N, Hq, Hk = case["B"], case["N"], case["Hq"], case["Hk"]
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    pos, start, n_max = _positions(case, r)
    s = {"case": case, "pos": None if pos is None else _i32(pos), "start": None if start is None else _i32(start)}
    # forward: from the projection's layout to [B, H, N, 64]; back: the other way round
    base, q, k = _views(case, Hq, Hk, dt, g)
    if case["back"]:
        s["q"], s["k"] = q.contiguous(), k.contiguous() if Hk else None
        s["y"], s["yq"], s["yk"] = base, q, k
        if base is None:
            s["yq"], s["yk"] = torch.zeros_like(q), torch.zeros_like(k) if Hk else None
        else:
            base.zero_()  # the gradient of the projection; the values' part comes from elsewhere
    else:
        s["q"], s["k"] = q, k
        s["yq"] = torch.zeros((B, Hq, N, D), device="cuda", dtype=dt)
        s["yk"] = torch.zeros((B, Hk, N, D), device="cuda", dtype=dt) if Hk else None
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        s["rope"] = fa.fib_attn_rope_create(
            n_max, rot_dim=case["R"], layout={"half": fa.FIB_ROPE_HALF, "interleaved": fa.FIB_ROPE_INTERLEAVED}[case["layout"]], base=BASE,
            scaling={"plain": fa.FIB_ROPE_PLAIN, "linear": fa.FIB_ROPE_LINEAR, "ntk": fa.FIB_ROPE_NTK, "yarn": fa.FIB_ROPE_YARN}[case["scaling"]],
            factor=case["factor"], n_train=1024)
    return s


def _lens(B, most):
    """Lengths from some of `most` up to it; among four or more a short one."""
    v = [max(1, most - (most * i) // (2 * B) - (i * 13) % 29) for i in range(B)]
    v[0] = most
    if B >= 4:
        v[1] = max(1, most // 9)
    return v


def _n_new(case):
    """What each sequence has just gained, no more than its length; among four or more one takes no part."""
    T = case["T"]
    n = [min(x, 1 + (i * 5) % T if case["path"] else T) for i, x in enumerate(_lens(case["B"], case["len"]))]
    if case["B"] >= 4:
        n[2] = 0
    return n


def _pages(r, lens, P, group, spare):
    """(table, refs): pages in any order, sequences in groups that share those of the first of them."""
    lens = np.asarray(lens)
    B, MP = len(lens), -(-int(lens.max()) // P) + 1
    b, j = np.arange(B)[:, None], np.arange(MP)
    lead = b - b % group
    held = np.where(b == lead, -(-lens[:, None] // P), 0)
    NP = int(held.sum()) + spare
    ids = r.permutation(NP)
    first = np.cumsum(held[:, 0]) - held[:, 0]
    table = np.where(j < -(-lens[:, None] // P), ids[np.minimum(first[lead] + j, NP - 1)], -1)
    return table, np.bincount(table[table >= 0], minlength=NP)


def _prepare_weigh(case, seed):
    L, B, Hq, H, T, P = (case[x] for x in ("L", "B", "Hq", "H", "T", "P"))
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    order = r.permutation(B)
    lens, n_new = np.asarray(_lens(B, case["len"]))[order], np.asarray(_n_new(case))[order]
    table, refs = _pages(r, lens, P, 1, 3)
    path = np.tile(np.arange(T), (B, 1))
    if case["path"]:  # the nodes of a root-to-node path, ascending
        taken = np.argsort(np.argsort(r.rand(B, T), axis=1), axis=1) < n_new[:, None]
        path = np.argsort(~taken, axis=1, kind="stable")
    rows = case["len"] + 5
    s = {"case": case, "q": _randn((L, B, Hq, T, D), dt, g), "k": _randn((L, len(refs), H, P, D), dt, g), "table": _i32(table),
         "lens": _i32(lens), "refs": _i32(refs), "n_new": _i32(n_new), "path": _i32(path), "first": torch.zeros(B, device="cuda", dtype=torch.int32),
         "weights": _randn((L, B, H, rows), torch.float32, g).square_().mul_(4.0 * Hq * T / (H * case["len"]))}  # of a few steps
    # the log-sum-exp of len scores N(0, 1), about
    s["lse"] = (torch.log(s["lens"].float()) + 0.5)[None, :, None, None] + 0.1 * _randn((L, B, Hq, T), torch.float32, g)
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        s["plan"] = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.0] * L, 12, max(int(lens.max()), 2), fa.FIB_MODE_MASK)
        s["cache"] = _own_cache(fa, s, dt)
        s["workspace"] = torch.empty(max(1, fa.fib_attn_cache_weigh_workspace_size(s["cache"], B, Hq, T)), device="cuda", dtype=torch.uint8)
    return s


def _own_cache(fa, s, dt):
    L, NP, H, P = s["k"].shape[:4]
    v = s.get("v")
    cache = fa.fib_attn_cache_create(L, H, P, NP, s["table"].shape[0], s["table"].shape[1], dt, k=s["k"],
                                     v=torch.empty_like(s["k"]) if v is None else v)
    cache.table.copy_(s["table"])
    cache.lens.copy_(s["lens"])
    cache.refs.copy_(s["refs"])
    return cache


def _keeps(case, lens):
    """How many rows each sequence keeps: the budget, a little less for some; a short sequence stays as it is."""
    low = case["sink"] + case["recent"]
    return [max(low, case["keep"] - (i * 3) % 17) for i in range(len(lens))]


def _group_lens(case):
    """Lengths of a group of sequences differ only behind what they share."""
    G = case["group"]
    v = _lens(-(-case["B"] // G), case["len"])
    return [max(1, v[b // G] - (b % G)) for b in range(case["B"])]


def _prepare_evict(case, seed):
    L, B, H, P = (case[x] for x in ("L", "B", "H", "P"))
    dt = TYPES[case["dtype"]]
    g, r = _gen(seed), np.random.RandomState(seed % (1 << 31))
    lens = _group_lens(case)
    spare = 3 + (0 if case["group"] == 1 else B * (-(-case["keep"] // P) + 1))
    table, refs = _pages(r, lens, P, case["group"], spare)
    NP, rows = len(refs), case["len"] + 3
    # accumulated weights: long-tailed, many of them equal (held to steps of 1/64)
    w = torch.floor(torch.exp(1.5 * _randn((L, B, H, rows), torch.float32, g)) * 64) / 64
    s = {"case": case, "k": _randn((L, NP, H, P, D), dt, g), "v": _randn((L, NP, H, P, D), dt, g), "table": _i32(table), "lens": _i32(lens),
         "refs": _i32(refs), "keep": _i32(_keeps(case, lens)), "before": w, "weights": w.clone(),
         "dropped": torch.zeros(B, device="cuda", dtype=torch.int32)}
    if own:
        from fibonacci_offset_sparse_gb300 import fib_attn as fa
        s["plan"] = fa.fib_attn_plan_create(fa.FIB_BASE_FIBONACCI, [1.0] * L, 12, max(max(lens), 2), fa.FIB_MODE_MASK)
        s["cache"] = _own_cache(fa, s, dt)
        s["meta"] = s["cache"].meta.clone()
        s["workspace"] = torch.empty(max(1, fa.fib_attn_cache_evict_workspace_size(s["cache"], rows)), device="cuda", dtype=torch.uint8)
    return s


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "weigh": _prepare_weigh, "evict": _prepare_evict}[case["op"]](case, seed)


# ------------------------------------------------------------------------------------------ plain forms
def _theta(case, device):
    """(frequencies of the R/2 pairs in 64 bits, amplitude)."""
    R, f = case["R"], case["factor"]
    m = torch.arange(R // 2, device=device, dtype=torch.float64)
    base = BASE * f ** (R / (R - 2)) if case["scaling"] == "ntk" and R > 2 else BASE
    theta = torch.pow(torch.tensor(base, device=device, dtype=torch.float64), -2 * m / R)
    if case["scaling"] == "linear":
        theta = theta / f
    if case["scaling"] == "yarn":  # pairs of few turns in the 1024 positions of training are stretched, those of many kept
        keep = ((1024 * theta / (2 * math.pi) - 1) / 31).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / f)
    return theta, 0.1 * math.log(f) + 1 if case["scaling"] == "yarn" else 1.0


def _plain_turn(x, c, s, case, out):
    """x [B, H, N, 64] turned by c, s [B, 1, N, R/2] into out."""
    R = case["R"]
    z = x.float()
    if case["layout"] == "half":
        a, b = z[..., :R // 2], z[..., R // 2:R]
        turned = torch.cat([a * c - b * s, a * s + b * c], -1)
    else:
        a, b = z[..., :R:2], z[..., 1:R:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    out[..., :R] = turned
    out[..., R:] = x[..., R:]


def _plain_rotary(s):
    case = s["case"]
    dev = s["q"].device
    at = torch.arange(case["N"], device=dev)[None]
    pos = s["pos"] if s["pos"] is not None else at if s["start"] is None else s["start"][:, None] + at
    theta, amp = _theta(case, dev)
    a = (pos.double()[..., None] * theta)[:, None]
    c, sn = (amp * torch.cos(a)).float(), (amp * torch.sin(a)).float()
    sn = -sn if case["back"] else sn
    _plain_turn(s["q"], c, sn, case, s["yq"])
    if s["k"] is not None:
        _plain_turn(s["k"], c, sn, case, s["yk"])
    return _rotary_out(s)


def _rotary_out(s):
    return [s["y"]] if s.get("y") is not None else [s["yq"]] + ([s["yk"]] if s["yk"] is not None else [])


def _rope(x, pos):
    """Rotate-half pairs (m, m + 32) of x by pos * 10000^(-m/32), the angle in 64 bits."""
    m = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * torch.pow(torch.tensor(BASE, device=x.device, dtype=torch.float64), -m / 32)
    c, s = torch.cos(a).float(), torch.sin(a).float()
    x1, x2 = x[..., :D // 2].float(), x[..., D // 2:].float()
    return torch.cat([x1 * c - x2 * s, x1 * s + x2 * c], dim=-1)


def _plain_weigh(s):
    c = s["case"]
    L, B, Hq, H, T, P = (c[x] for x in ("L", "B", "Hq", "H", "T", "P"))
    dev = s["q"].device
    lens, n, G = s["lens"].long(), s["n_new"].long(), Hq // H
    i = torch.arange(T, device=dev)
    pos = (lens - n)[:, None] + i  # [B, T]
    node = s["path"].long()[None, :, None, :, None]
    q = torch.gather(s["q"], 3, node.expand(L, B, Hq, T, D))
    lse = torch.gather(s["lse"], 3, node[..., 0].expand(L, B, Hq, T))
    q = _rope(q, pos[:, None, :]).view(L, B, H, G * T, D)
    table = s["table"].long().clamp(min=0)
    most = c["len"]
    page = table[:, :-(-most // P)]
    k = s["k"][:, page].permute(0, 1, 3, 2, 4, 5).reshape(L, B, H, -1, D)[..., :most, :].float()
    sc = q @ k.transpose(-1, -2) / 8
    r = torch.arange(most, device=dev)
    sees = (r <= pos[..., None]) & (i < n[:, None])[..., None]  # [B, T, rows]
    w = torch.exp(sc - lse.reshape(L, B, H, G * T, 1)).view(L, B, H, G, T, most)
    w = torch.where(sees[:, None, None], w, torch.zeros((), device=dev)).sum((3, 4))
    first = s["first"].long() if c["set"] else lens - n
    old = s["weights"][..., :most]
    new = torch.where(r < first[:, None, None], old, torch.zeros((), device=dev)) + w
    live = (r < lens[:, None]) & (n > 0)[:, None]
    s["weights"][..., :most] = torch.where(live[:, None], new, old)
    return [s["weights"]]


def _plain_evict(s):
    c = s["case"]
    L, B, H, P = (c[x] for x in ("L", "B", "H", "P"))
    dev = s["k"].device
    w = s["weights"]
    w.copy_(s["before"])  # a pass starts where the last one did
    lens, keep, refs, table = s["lens"].long(), s["keep"].long(), s["refs"].long(), s["table"].long()
    cut = lens > keep
    most, R = c["len"], w.shape[-1]
    r = torch.arange(most, device=dev)
    # the rows kept, in order: rank all rows with the first and the last on top, then the heaviest; equal ones as they lie
    inside = (r >= c["sink"]) & (r < (lens - c["recent"])[:, None])
    score = torch.where(inside[:, None], w[..., :most], torch.tensor(math.inf, device=dev))
    score = torch.where((r < lens[:, None])[:, None], score, torch.tensor(-math.inf, device=dev))
    rank = torch.argsort(torch.argsort(score, dim=-1, descending=True, stable=True), dim=-1)
    stays = rank < keep[:, None, None]
    src = torch.argsort((~stays).to(torch.uint8), dim=-1, stable=True)[..., :int(keep.max())]  # [L, B, H, j]: the row that comes to j
    # pages: shared ones that are written are replaced by free ones, those behind the new length are given back
    j = torch.arange(table.shape[1], device=dev)
    had, has = (lens + P - 1) // P, (keep + P - 1) // P
    same = torch.clamp(has, max=c["sink"] // P)
    written = cut[:, None] & (j >= same[:, None]) & (j < has[:, None])
    shared = written & (refs[table.clamp(min=0)] > 1)
    gone = cut[:, None] & (j >= has[:, None]) & (j < had[:, None])
    free = (refs == 0).nonzero().flatten()
    taken = free[:int(shared.sum())]
    now = table.clone()
    now[shared] = taken  # in the order of sequences, then of pages
    now[gone] = -1
    left = torch.cat([table[shared], table[gone]])
    refs = refs.index_add(0, left, -torch.ones_like(left))
    refs[taken] = 1
    # rows
    jb = torch.arange(src.shape[-1], device=dev)
    l, b, h, d = ((jb < keep[:, None]) & (jb >= (same * P)[:, None]) & cut[:, None])[None, :, None].expand(src.shape).nonzero(as_tuple=True)
    from_ = src[l, b, h, d]
    p0, p1 = table[b, from_ // P], now[b, d // P]
    k, v = s["k"], s["v"]
    k_rows, v_rows = _rope(k[l, p0, h, from_ % P], d - from_), v[l, p0, h, from_ % P]
    k_rows = torch.where((d == from_)[:, None], k[l, p0, h, from_ % P].float(), k_rows)
    k[l, p1, h, d % P] = k_rows.to(k.dtype)
    v[l, p1, h, d % P] = v_rows
    w[l, b, h, d] = s["before"][l, b, h, from_]
    dropped = s["dropped"]
    dropped.copy_(torch.where(cut, lens - keep, 0))
    return [k, v, w, now.int(), torch.where(cut, keep, lens).int(), refs.int(), dropped]


def _run_own(s):
    from fibonacci_offset_sparse_gb300 import fib_attn as fa
    c = s["case"]
    if c["op"] == "rotary":
        fa.fib_attn_rotary(s["rope"], s["q"], s["k"], pos=s["pos"], start=s["start"], transpose=c["back"], q_out=s["yq"], k_out=s["yk"])
        return _rotary_out(s)
    if c["op"] == "weigh":
        fa.fib_attn_cache_weigh(s["plan"], s["cache"], s["q"], s["lse"], s["n_new"], s["weights"], path=s["path"] if c["path"] else None,
                                first=s["first"] if c["set"] else None, workspace=s["workspace"])
        return [s["weights"]]
    cache = s["cache"]
    cache.meta.copy_(s["meta"])  # back to the tables and weights as they stood: a pass starts where the last one did
    s["weights"].copy_(s["before"])
    s["dropped"].zero_()
    fa.fib_attn_cache_evict(s["plan"], cache, s["weights"], s["keep"], c["sink"], c["recent"], dropped=s["dropped"], workspace=s["workspace"])
    return [cache.k, cache.v, s["weights"], cache.table, cache.lens, cache.refs, s["dropped"]]


def run(state):
    if own:
        return _run_own(state)
    return {"rotary": _plain_rotary, "weigh": _plain_weigh, "evict": _plain_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op = case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "rotary":
        rows = case["B"] * case["N"] * (case["Hq"] + case["Hk"])
        at = {"none": 0, "start": 4 * case["B"], "packed": 4 * case["B"] * case["N"]}[case["pos"]]
        return {"bytes": rows * 2 * D * es + at, "flops": rows * case["R"] * 3}
    L, B, H = case["L"], case["B"], case["H"]
    if op == "weigh":
        G = case["Hq"] // H
        lens, n = _lens(B, case["len"]), _n_new(case)
        rows = sum(x for x, y in zip(lens, n) if y)
        pairs = sum(y * (x - y) + y * (y + 1) // 2 for x, y in zip(lens, n))  # token i of the last n sees all rows up to its own
        old = 0 if case["set"] else 4 * rows  # weights that are set are not read
        return {"bytes": L * H * (rows * (D * es + 4) + old) + L * sum(n) * case["Hq"] * (D * es + 4),
                "flops": L * H * G * pairs * (2 * D + 3)}
    lens = _group_lens(case)
    keeps = _keeps(case, lens)
    cut = [(x, k) for x, k in zip(lens, keeps) if x > k]
    moved = sum(k - min(k, case["sink"]) for _, k in cut)  # what stands before the first row that leaves stays: next to nothing
    weighed = sum(x - case["sink"] - case["recent"] for x, _ in cut)
    return {"bytes": L * H * (moved * 4 * D * es + weighed * 4 + moved * 8), "flops": L * H * moved * D * 3}


# ------------------------------------------------------------------------------------------ 64 bits
def _exact_rotary(s, case):
    R, f = case["R"], case["factor"]
    N, dev = case["N"], s["q"].device
    if s["pos"] is not None:
        pos = s["pos"].double()
    else:
        pos = torch.arange(N, device=dev, dtype=torch.float64).expand(case["B"], N)
        pos = pos if s["start"] is None else pos + s["start"].double()[:, None]
    freq = [BASE ** (-2.0 * m / R) for m in range(R // 2)]
    if case["scaling"] == "linear":
        freq = [x / f for x in freq]
    elif case["scaling"] == "ntk" and R > 2:
        freq = [x * f ** (-2.0 * m / (R - 2)) for m, x in enumerate(freq)]
    elif case["scaling"] == "yarn":
        ramp = [min(1.0, max(0.0, (1024 * x / (2 * math.pi) - 1.0) / 31.0)) for x in freq]
        freq = [x * g + x / f * (1 - g) for x, g in zip(freq, ramp)]
    amp = 1.0 + 0.1 * math.log(f) if case["scaling"] == "yarn" else 1.0
    turn = pos[:, None, :, None] * torch.tensor(freq, device=dev, dtype=torch.float64) * (-1.0 if case["back"] else 1.0)
    turn = torch.polar(torch.full_like(turn, amp), turn)
    lo, hi = (slice(0, R // 2), slice(R // 2, R)) if case["layout"] == "half" else (slice(0, R, 2), slice(1, R, 2))
    whole = None if s.get("y") is None else s["y"].double()

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
        out = x.clone(memory_format=torch.contiguous_format)
        out[..., lo], out[..., hi] = z.real, z.imag
        return out

    into = [turned(x) for x in (s["q"], s["k"]) if x is not None]
    if whole is None:
        return into
    heads = torch.cat(into, 1).transpose(1, 2)
    whole[:, :, :heads.shape[2]] = heads
    return [whole]


def _turned(x, pos):
    """x [..., 64] as 32 complex numbers turned by pos: back as 64 reals, in 64 bits."""
    x = x.double()
    z = torch.complex(x[..., :32].contiguous(), x[..., 32:].contiguous())
    m = torch.arange(32, device=x.device, dtype=torch.float64)
    a = pos.double()[..., None] * torch.exp(-m / 32 * math.log(BASE))
    z = z * torch.polar(torch.ones_like(a), a)
    return torch.cat([z.real, z.imag], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s, case)
    P, H, L = case["P"], case["H"], case["L"]
    lens, table = s["lens"].tolist(), s["table"].tolist()
    w = s["weights"].double()
    if case["op"] == "weigh":
        G = case["Hq"] // H
        for b, n in enumerate(s["n_new"].tolist()):
            if not n:
                continue
            length = lens[b]
            pages = torch.tensor(table[b][:-(-length // P)], device="cuda")
            nodes = s["path"][b, :n].long()
            at = torch.arange(length - n, length, device="cuda")
            hidden = torch.arange(length, device="cuda") > at[:, None]
            for layer in range(L):
                K = s["k"][layer, pages].double().transpose(0, 1).reshape(H, -1, D)[:, :length]
                q = _turned(s["q"][layer, b][:, nodes], at).view(H, G, n, D)
                sc = torch.einsum("hgtd,hkd->hgtk", q, K) / 8 - s["lse"][layer, b][:, nodes].double().view(H, G, n, 1)
                given = torch.exp(sc.masked_fill(hidden, -math.inf)).sum((1, 2))
                from_ = 0 if case["set"] else length - n
                w[layer, b, :, from_:length] = 0
                w[layer, b, :, :length] += given
        return [w]
    keep, refs = s["keep"].tolist(), s["refs"].tolist()
    k0, v0, held = s["k"].double(), s["v"].double(), list(refs)
    k, v = k0.clone(), v0.clone()
    dropped, now, new = [0] * len(lens), list(lens), [list(x) for x in table]
    free = iter([p for p, x in enumerate(refs) if not x])
    before = s["before"]
    for b, length in enumerate(lens):
        n = keep[b]
        if length <= n:
            continue
        dropped[b], now[b] = length - n, n
        for j in range(-(-length // P)):
            page = table[b][j]
            if j >= -(-n // P):
                new[b][j] = -1
                refs[page] -= 1
            elif j >= case["sink"] // P and held[page] > 1:
                new[b][j] = next(free)
                refs[new[b][j]] = 1
                refs[page] -= 1
        end = length - case["recent"]
        # the middle rows by weight, heaviest first, the first of equal ones first: weight and place in one number
        mid = before[:, b, :, case["sink"]:end].double().cpu().numpy()
        order = np.argsort(-mid, axis=-1, kind="stable")[..., :n - case["sink"] - case["recent"]] + case["sink"]
        edge = np.broadcast_to(np.concatenate([np.arange(case["sink"]), np.arange(end, length)]), order.shape[:-1] + (case["sink"] + case["recent"],))
        src = torch.from_numpy(np.sort(np.concatenate([order, edge], -1), axis=-1).astype(np.int64)).cuda()  # [L, H, n]
        dst = torch.arange(n, device="cuda")
        old_page, new_page = torch.tensor(table[b], device="cuda")[src // P], torch.tensor(new[b], device="cuda")[dst // P]
        li, hi = torch.arange(L, device="cuda")[:, None, None], torch.arange(H, device="cuda")[:, None]
        k[li, new_page, hi, dst % P] = _turned(k0[li, old_page, hi, src % P], dst - src)
        v[li, new_page, hi, dst % P] = v0[li, old_page, hi, src % P]
        w[:, b, :, :n] = torch.gather(before[:, b].double(), -1, src)
    i32 = lambda x: np.asarray(x, np.int32)  # noqa: E731
    return [k, v, w, i32(new), i32(now), i32(refs), i32(dropped)]
