"""The operators behind a verified tree, as timed and compared work.

sample:  tokens drawn from logits with temperature, top-k, top-p and min-p, from given random numbers
accept:  the walk down each tree along the tokens drawn at its nodes, and the keys and values of the path moved to
         where the next tokens follow them
weights: a chunk's attention weights added to what each cached position has gathered
evict:   per head the positions that have gathered most stay in the cache, in their order

``own = False`` computes them in plain torch operations, ``own = True`` through the package.  A case is a dict of
plain values; its lengths follow from those values alone, the numbers in them from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _sample(name=None, **over):
    c = dict(op="sample", dtype="bf16", B=1, R=1, V=151936, pad=0, top_k=False, top_p=False, min_p=False, spread=2.0)
    c.update(over)
    return dict(c, name=name) if name else c


def _cached(op, name, over):
    c = dict(op=op, dtype="bf16", B=1, ctx=1024, Hkv=8, D=128, page=64)
    c.update(over)
    return dict(c, name=name) if name else c


def _accept(name=None, **over):
    return _cached("accept", name, dict(dict(N=78, depth=8), **over))


def _weights(name=None, **over):
    return _cached("weights", name, dict(dict(n=1, Hq=32, tree=0), **over))


def _evict(name=None, **over):
    return _cached("evict", name, dict(dict(keep=512, first=4, last=64), **over))


def listed():
    return [
        # the next token of one sequence, with the settings of a chat
        _sample("sample_one_token", top_k=True, top_p=True),
        # the 79 rows of 64 verified trees, each sequence with a top-p of its own: what is kept reaches far down
        _sample("sample_trees_top_p", dtype="f16", B=64, R=79, V=32000, top_p=True),
        # the 497 rows of four wide trees over a large vocabulary, all three limits
        _sample("sample_wide_trees", B=4, R=497, top_k=True, top_p=True, min_p=True),
        # 500 rows in 32 bits with the temperature alone
        _sample("sample_f32_all", dtype="f32", B=100, R=5, V=32000),
        # one tree of 78 nodes
        _accept("accept_one_tree"),
        # 64 trees of 496 nodes, 16 deep, in 16-token pages
        _accept("accept_wide_trees", B=64, N=496, depth=16, ctx=2048, page=16),
        # one token of one sequence over 4098 positions
        _weights("weights_one_token", ctx=4097),
        # a decode step of 64 sequences of about 6000 tokens
        _weights("weights_decode_batch", B=64, ctx=8192),
        # 64 trees of 78 nodes behind their roots over about 1500 tokens each
        _weights("weights_trees", B=64, n=79, ctx=2048, tree=78, page=16),
        # one long sequence brought back to half of its length
        _evict("evict_long", ctx=32768, keep=16384, page=128),
        # 32 sequences of about 6000 tokens brought back to 2048
        _evict("evict_batch", dtype="f16", B=32, ctx=8192, keep=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    worst = {}
    for c in listed():
        seen = worst.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for key, w in work(c).items():
            seen[key] = max(seen[key], w)
    op = rng.choice(["sample", "sample", "accept", "weights", "weights", "evict", "evict"])
    while True:
        if op == "sample":
            c = _sample(dtype=rng.choice(["bf16", "f16", "f32"]), B=_log_int(rng, 1, 256), R=_log_int(rng, 1, 497),
                        V=rng.choice([32000, 151936, _log_int(rng, 100, 200000)]), pad=rng.choice([0, 0, 8, 61]),
                        top_k=rng.random() < 0.5, top_p=rng.random() < 0.5, min_p=rng.random() < 0.3,
                        spread=rng.choice([0.5, 1.0, 2.0, 3.0]))
            if c["B"] * c["R"] * c["V"] > 1.7e8:
                continue
        else:
            common = dict(dtype=rng.choice(["bf16", "f16"]), B=_log_int(rng, 1, 128), Hkv=rng.choice([1, 2, 4, 8]),
                          D=rng.choice([64, 80, 96, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                          ctx=_log_int(rng, 32, 32768))
            if op == "accept":
                N = _log_int(rng, 1, 496)
                c = _accept(N=N, depth=rng.randint(1, min(N, 24)), **common)
            elif op == "weights":
                tree = rng.choice([0, 0, _log_int(rng, 5, 496)])
                c = _weights(n=tree + 1 if tree else rng.choice([1, 1, _log_int(rng, 2, 512)]), tree=tree,
                             Hq=common["Hkv"] * rng.choice([1, 3, 4, 7, 8]), **common)
            else:
                keep = _log_int(rng, 16, common["ctx"])
                first = rng.randint(0, min(8, keep // 2))
                c = _evict(keep=keep, first=first, last=rng.randint(0, keep - first), **common)
        w = work(c)
        # the caches are held several times over while cases are compared
        cache = 4 * c["B"] * (c["ctx"] + 512) * c["Hkv"] * c["D"] if "ctx" in c else 0
        if all(w[key] <= worst[op][key] for key in w) and cache < 4e9:
            return c


def _context(c):
    """Each sequence's tokens in the cache: the first has all of ctx, the others down to half of it."""
    return [c["ctx"] - (b * 7919) % (c["ctx"] // 2 + 1) for b in range(c["B"])]


def _chunks(c):
    """Each sequence's new tokens: all n of a tree and of a single sequence, else down to half of n."""
    if c["tree"] or c["n"] == 1:
        return [c["n"]] * c["B"]
    return [c["n"] - (b * 104729) % (c["n"] // 2 + 1) for b in range(c["B"])]


def _accepted(c):
    """The nodes accepted in each tree."""
    return [(b * 7919 + c["depth"] // 2) % (c["depth"] + 1) for b in range(c["B"])]


def _depths(N, depth):
    """The depth of each of N nodes, numbered depth by depth, all depths about equally wide."""
    return [1 + i * depth // N for i in range(N)]


def _tree_depths(N):
    width = N // 16 + 4
    return [1 + i // width for i in range(N)]


def work(case):
    c = case
    if c["op"] == "sample":
        rows = c["B"] * c["R"]
        return {"bytes": rows * (c["V"] * BYTES[c["dtype"]] + 12) + 16 * c["B"], "flops": 4 * rows * c["V"]}
    row = 2 * c["Hkv"] * c["D"] * BYTES[c["dtype"]]          # a position's keys and values
    if c["op"] == "accept":
        moved = 2 * row * sum(_accepted(c))
        return {"bytes": moved + c["B"] * 4 * (3 * c["N"] + 2 * c["depth"] + 6), "flops": 2 * c["B"] * c["N"]}
    if c["op"] == "evict":
        # a kept row beyond the protected ones moves; the caches' other rows stay
        kept = [min(x, c["keep"]) if x > c["keep"] else 0 for x in _context(c)]
        moved = sum(max(k - c["first"], 0) for k in kept)
        scores = sum(8 * x for x, k in zip(_context(c), kept) if k)
        return {"bytes": 2 * row * moved + c["Hkv"] * (scores + 4 * sum(kept)), "flops": 2 * c["Hkv"] * sum(_context(c))}
    rows = sum(x + n for x, n in zip(_context(c), _chunks(c)))
    tokens = sum(_chunks(c))
    pairs = 0
    for x, n in zip(_context(c), _chunks(c)):
        lead = n - c["tree"]
        pairs += lead * x + lead * (lead + 1) // 2 + c["tree"] * (x + lead) + sum(_tree_depths(c["tree"]))
    return {"bytes": rows * (row // 2 + 8 * c["Hkv"]) + tokens * c["Hq"] * (c["D"] * 2 + 4),
            "flops": (2 * c["D"] + 2) * c["Hq"] * pairs}


# ------------------------------------------------------------------ inputs

def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _trees(depths, B, rng):
    """parents [B, N] of random trees with those depths, and the nodes' packed ancestor-or-self masks."""
    depth, N = np.array(depths), len(depths)
    parents = np.full((B, N), -1, np.int32)
    bits = np.zeros((B, N, 32 * ((N + 31) // 32)), np.uint8)
    first = {d: int(np.argmax(depth == d)) for d in set(depth.tolist())}
    for i in range(N):
        d = int(depth[i])
        if d > 1:
            parents[:, i] = rng.integers(first[d - 1], first[d], size=B)
            bits[:, i] = bits[np.arange(B), parents[:, i]]
        bits[:, i, i] = 1
    return parents, np.packbits(bits, axis=-1, bitorder="little").view(np.int32)


def _paths(c, parents, rng):
    """Each tree's accepted path: a random node of the accepted depth and what lies above it, from the top."""
    depth = np.array(_depths(c["N"], c["depth"]))
    paths = []
    for b, a in enumerate(_accepted(c)):
        path, i = [], int(rng.choice(np.nonzero(depth == a)[0])) if a else -1
        while i >= 0:
            path.append(i)
            i = int(parents[b, i])
        paths.append(path[::-1])
    return paths


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B = c["B"]
    s = {"case": c}
    if c["op"] == "sample":
        return _prepare_sample(c, s, rng, gen)
    dt, P, D, Hkv = DTYPES[c["dtype"]], c["page"], c["D"], c["Hkv"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    ctx = _context(c)
    new = _chunks(c) if c["op"] == "weights" else [c.get("N", 0) + 1] * B
    need = [(x + n + P - 1) // P for x, n in zip(ctx, new)]
    total = sum(need) + 3                       # pages in random order, a few of them nobody's
    order = rng.permutation(total)
    table, at = np.zeros((B, max(need)), np.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    s.update(ctx=ctx, new=new, pages=_gpu(table), lengths=_gpu(np.array(ctx, np.int32)))
    s["k_cache"] = normal(total, P, Hkv, D)
    if c["op"] != "weights":
        s["v_cache"] = normal(total, P, Hkv, D)
    if c["op"] == "accept":
        N = c["N"]
        parents, _ = _trees(_depths(N, c["depth"]), B, rng)
        # the children of a node carry distinct tokens; the nodes' numbers in a random order serve
        tokens = np.argsort(rng.random((B, N)), axis=1).astype(np.int32) + 100
        picks = rng.integers(0, 100, size=(B, N + 1)).astype(np.int32)
        for b, path in enumerate(_paths(c, parents, rng)):
            at = 0
            for i in path:
                picks[b, at] = tokens[b, i]
                at = i + 1
        s.update(picks=_gpu(picks), tokens=_gpu(tokens), parents=_gpu(parents))
        return s
    width = table.shape[1] * P
    # weight gathered so far: most positions have little, some a lot, as the sums of many softmax rows have it
    s["scores"] = torch.rand((B, Hkv, width), generator=gen, device="cuda").pow_(6.0).mul_(4.0)
    if c["op"] == "evict":
        return s
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s["starts"], s["q"] = _gpu(starts), normal(int(starts[-1]), c["Hq"], D)
    if c["tree"]:
        s["mask"] = _gpu(_trees(_tree_depths(c["tree"]), B, rng)[1])
    # the log of each row's sum, which the attention before this step has returned
    s["lse"] = torch.cat([x.logsumexp(-1) for x in _scores(s)])
    return s


def _prepare_sample(c, s, rng, gen):
    B, R, V = c["B"], c["R"], c["V"]
    # a smooth part, and per row some tokens far above it, as a model's logits have them
    z = torch.randn((B, R, V + c["pad"]), generator=gen, device="cuda", dtype=torch.float32).mul_(c["spread"])
    ids = torch.randint(0, V, (B, R, 24), generator=gen, device="cuda")
    z.scatter_add_(2, ids, torch.rand((B, R, 24), generator=gen, device="cuda") * 14.0)
    s["logits"] = z.to(DTYPES[c["dtype"]])[..., :V]
    s["uniforms"] = torch.rand((B, R), generator=gen, device="cuda")
    heat = rng.uniform(0.6, 1.2, B).astype(np.float32)
    heat[rng.random(B) < 0.1] = 0.0             # some sequences are decoded greedily
    s["temperature"] = _gpu(heat)
    s["top_k"] = _gpu(rng.choice(np.array([20, 40, 50, 100, 1000, 0], np.int32), B)) if c["top_k"] else None
    s["top_p"] = _gpu(rng.uniform(0.7, 0.99, B).astype(np.float32)) if c["top_p"] else None
    s["min_p"] = _gpu(rng.uniform(0.01, 0.1, B).astype(np.float32)) if c["min_p"] else None
    return s


# ------------------------------------------------------------------- calls

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return {"sample": _own_sample, "accept": _own_accept, "weights": _own_weights,     "evict": _own_evict}[op](s)
    return {"sample": _plain_sample, "accept": _plain_accept, "weights": _plain_weights, "evict": _plain_evict}[op](s)


def _own_sample(s):
    import draft_tree_construction_gb300 as dart
    out = dart.sample_logits(s["logits"], s["uniforms"], temperature=s["temperature"], top_k=s["top_k"],
                             top_p=s["top_p"], min_p=s["min_p"])
    return out["tokens"], out["probs"]


def _own_accept(s):
    import draft_tree_construction_gb300 as dart
    out = dart.tree_accept(s["picks"], s["tokens"], s["parents"], s["case"]["depth"])
    lengths = dart.kv_keep(s["k_cache"], s["v_cache"], s["pages"], s["lengths"], out["path"], out["counts"])
    return out["path"], out["counts"], out["tokens"], s["k_cache"], s["v_cache"], lengths


def _own_weights(s):
    import draft_tree_construction_gb300 as dart
    return dart.attention_weights(s["q"], s["k_cache"], s["pages"], s["lengths"], s["starts"], s["lse"], s["scores"],
                                  mask=s.get("mask"))


def _own_evict(s):
    import draft_tree_construction_gb300 as dart
    c = s["case"]
    out = dart.kv_evict(s["k_cache"], s["v_cache"], s["pages"], s["lengths"], s["scores"], c["keep"],
                        first=c["first"], last=c["last"])
    return s["k_cache"], s["v_cache"], s["scores"], out["lengths"], out["index"]


def _plain_sample(s):
    """64 bits: which token a random number falls on is a matter of the last bits of long sums."""
    V = s["logits"].shape[-1]
    z, ids = s["logits"].double().sort(dim=-1, descending=True, stable=True)
    heat = s["temperature"].double()[:, None, None]
    w = torch.exp((z - z[..., :1]) / torch.where(heat > 0, heat, 1.0))
    rank = torch.arange(V, device="cuda")
    limit = torch.where(heat > 0, V, 1)
    if s["top_k"] is not None:
        k = s["top_k"][:, None, None]
        limit = torch.minimum(limit, torch.where(k > 0, k, V))
    w = torch.where(rank < limit, w, 0.0)
    total = w.cumsum(-1)
    kept = rank < limit
    if s["top_p"] is not None:
        # a token stays while those before it have not reached the share
        kept = kept & ((rank == 0) | (total - w < s["top_p"].double()[:, None, None] * total[..., -1:]))
    if s["min_p"] is not None:
        kept = kept & (w >= s["min_p"].double()[:, None, None])
    w = torch.where(kept, w, 0.0)
    total = w.cumsum(-1)
    at = (total <= s["uniforms"].double()[..., None] * total[..., -1:]).sum(-1, keepdim=True)
    at = torch.minimum(at, kept.sum(-1, keepdim=True) - 1)
    return ids.gather(-1, at)[..., 0].int(), (w.gather(-1, at) / total[..., -1:])[..., 0].float()


def _plain_accept(s):
    c = s["case"]
    B = c["B"]
    at = torch.zeros(B, dtype=torch.int64, device="cuda")        # the row of the node reached, 0 for the root
    on = torch.ones(B, dtype=torch.bool, device="cuda")
    path, tokens = [], []
    for _ in range(c["depth"] + 1):
        pick = s["picks"].gather(1, at[:, None])
        path.append(torch.where(on, at, -1))
        tokens.append(torch.where(on, pick[:, 0], -1))
        child = (s["parents"] == at[:, None] - 1) & (s["tokens"] == pick)
        on = on & child.any(1)
        at = torch.where(on, child.int().argmax(1) + 1, at)
    path = torch.stack(path, 1).int()
    counts = (path >= 0).sum(1).int()
    # a chunk's first row is the root, node i's is row i + 1; the path's rows move up behind the root
    lengths = s["lengths"].long()
    seq, i = torch.nonzero(path >= 0, as_tuple=True)
    source = _rows(s, seq, lengths[seq] + path[seq, i])
    target = _rows(s, seq, lengths[seq] + i)
    s["k_cache"][target] = s["k_cache"][source]
    s["v_cache"][target] = s["v_cache"][source]
    return path, counts, torch.stack(tokens, 1).int(), s["k_cache"], s["v_cache"], s["lengths"] + counts


def _rows(s, seq, position):
    page = s["case"]["page"]
    return s["pages"][seq, position // page].long(), position % page


def _unpack(words, count):
    """int32 [..., W] -> 0 / 1 int32 [..., count], the lowest bit of each word first."""
    shift = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words.unsqueeze(-1) >> shift) & 1).flatten(-2)[..., :count]


def _scores(s):
    """Per sequence the scaled products [n, Hq, S] in 32 bits, -inf where a row does not see."""
    c = s["case"]
    Hq, Hkv, D, P, N = c["Hq"], c["Hkv"], c["D"], c["page"], c["tree"]
    at = 0
    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        S, lead = x + n, n - N
        key = s["k_cache"][s["pages"][b, :(S + P - 1) // P].long()].flatten(0, 1)[:S].float()
        seen = torch.arange(S, device="cuda")[None, :] <= x + torch.arange(n, device="cuda")[:, None]
        if N:
            seen[lead:, x + lead:] = _unpack(s["mask"][b], N) == 1
        q = s["q"][at:at + n].float().view(n, Hkv, Hq // Hkv, D)
        z = torch.einsum("nhgd,shd->nhgs", q, key).flatten(1, 2) * (1.0 / math.sqrt(D))
        yield z.masked_fill_(~seen[:, None, :], -math.inf)
        at += n


def _plain_weights(s):
    c, at = s["case"], 0
    for b, z in enumerate(_scores(s)):
        n, Hq, S = z.shape
        p = z.sub_(s["lse"][at:at + n, :, None]).exp_()
        s["scores"][b, :, :S] += p.view(n, c["Hkv"], Hq // c["Hkv"], S).sum((0, 2))
        at += n
    return s["scores"]


def _plain_evict(s):
    c = s["case"]
    B, Hkv, width = s["scores"].shape
    keep, first, last = c["keep"], c["first"], c["last"]
    lengths = s["lengths"].long()
    position = torch.arange(width, device="cuda")
    inside = position < lengths[:, None]
    sure = inside & ((position < first) | (position >= lengths[:, None] - last))
    x = torch.where(sure[:, None], math.inf, s["scores"])
    x = torch.where(inside[:, None], x, -math.inf)
    # the first `keep` of the scores in descending order (the earlier position first where they are equal), by position
    best = x.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < lengths[:, None, None], best, width).sort(dim=-1).values
    count = torch.minimum(lengths, torch.tensor(keep, device="cuda"))
    seq, head, i = torch.nonzero(best < width, as_tuple=True)
    old = best[seq, head, i]
    source, target = _rows(s, seq, old), _rows(s, seq, i)
    for cache in (s["k_cache"], s["v_cache"]):
        cache[target[0], target[1], head] = cache[source[0], source[1], head]
    moved = s["scores"][seq, head, old]
    s["scores"].masked_fill_((inside & (position >= count[:, None]))[:, None], 0.0)
    s["scores"][seq, head, i] = moved
    index = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    index[seq, head, i] = old.int()
    return s["k_cache"], s["v_cache"], s["scores"], count.int(), index


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    """What run returns, from the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    return {"sample": _exact_sample, "accept": _exact_accept, "weights": _exact_weights, "evict": _exact_evict}[case["op"]](s)


def _exact_sample(s):
    B, R, V = s["logits"].shape
    tokens = torch.zeros((B, R), dtype=torch.int32, device="cuda")
    probs = torch.zeros((B, R), dtype=torch.float64, device="cuda")
    for b in range(B):
        heat = float(s["temperature"][b])
        k, p, m = (s[key][b].item() if s[key] is not None else None for key in ("top_k", "top_p", "min_p"))
        for r in range(R):
            z, order = torch.sort(s["logits"][b, r].double(), descending=True, stable=True)
            if heat <= 0:
                tokens[b, r], probs[b, r] = order[0], 1.0
                continue
            w = torch.exp((z - z[0]) / heat)[:k if k else V]
            if p is not None:
                reached = torch.cumsum(w, 0) >= p * torch.sum(w)
                short = w[:max(1, len(w) - int(reached.sum()) + 1)]
            else:
                short = w
            if m is not None:
                short = short[short >= m] if m <= 1.0 else short[:1]
            part = torch.cumsum(short, 0)
            i = min(int((part <= float(s["uniforms"][b, r]) * part[-1]).sum()), len(part) - 1)
            tokens[b, r], probs[b, r] = order[i], short[i] / part[-1]
    return tokens, probs


def _exact_accept(s):
    c, P = s["case"], s["case"]["page"]
    B, width = c["B"], c["depth"] + 1
    picks, tokens, parents, table = (s[key].cpu().numpy() for key in ("picks", "tokens", "parents", "pages"))
    path, counts, out = (np.full(shape, -1, np.int32) for shape in ((B, width), (B,), (B, width)))
    caches = [s["k_cache"].clone(), s["v_cache"].clone()]
    for b in range(B):
        children = {(int(p), int(t)): i for i, (p, t) in reversed(list(enumerate(zip(parents[b], tokens[b]))))}
        at, n = -1, 0
        while True:
            path[b, n], out[b, n], n = at + 1, picks[b, at + 1], n + 1
            if (at, int(picks[b, at + 1])) not in children:
                break
            at = children[at, int(picks[b, at + 1])]
        counts[b] = n
        for i in range(n):
            old, new = s["ctx"][b] + int(path[b, i]), s["ctx"][b] + i
            for cache, before in zip(caches, (s["k_cache"], s["v_cache"])):
                cache[int(table[b, new // P]), new % P] = before[int(table[b, old // P]), old % P]
    return (_gpu(path), _gpu(counts), _gpu(out), caches[0].double(), caches[1].double(),
            s["lengths"] + _gpu(counts))


def _exact_weights(s):
    c = s["case"]
    if work(c)["flops"] > 5e11:                 # beyond about 20 seconds of 64-bit products
        return None
    out, at, G, P, N = s["scores"].double(), 0, c["Hq"] // c["Hkv"], c["page"], c["tree"]
    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        slot = torch.arange(x + n, device="cuda")
        page, lead = s["pages"][b].long()[slot // P], n - N
        hidden = slot[None, :] > x + torch.arange(n, device="cuda")[:, None]
        if N:
            j = torch.arange(N, device="cuda")
            hidden[lead:, x + lead:] = ((s["mask"][b].long()[:, j // 32] >> (j % 32)) & 1) == 0
        for g in range(c["Hq"]):
            key = s["k_cache"][page, slot % P, g // G].double()
            z = (s["q"][at:at + n, g].double() @ key.T) / math.sqrt(c["D"])
            # the weights as the rows' sums that the caller hands over make them
            p = torch.exp(z - s["lse"][at:at + n, g].double()[:, None])
            out[b, g // G, :x + n] += p.masked_fill(hidden, 0.0).sum(0)
        at += n
    return out


def _exact_evict(s):
    c = s["case"]
    B, Hkv, _ = s["scores"].shape
    keep, first, last, P = c["keep"], c["first"], c["last"], c["page"]
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    scores = s["scores"].double()
    index = np.full((B, Hkv, keep), -1, np.int32)
    host, lengths = s["scores"].cpu().numpy(), []
    for b, x in enumerate(s["ctx"]):
        n = min(x, keep)
        lengths.append(n)
        table = s["pages"][b].long()
        for h in range(Hkv):
            free = np.arange(first, max(x - last, first)) if x > keep else np.arange(0)
            rest = np.concatenate([np.arange(min(first, x)), np.arange(max(x - last, first), x)]) if x > keep else np.arange(x)
            best = free[np.argsort(-host[b, h, free], kind="stable")][:n - len(rest)]
            index[b, h, :n] = np.sort(np.concatenate([rest, best]))
            old, new = _gpu(index[b, h, :n].astype(np.int64)), torch.arange(n, device="cuda")
            for cache, before in zip(caches, (s["k_cache"], s["v_cache"])):
                cache[table[new // P], new % P, h] = before[table[old // P], old % P, h].double()
            scores[b, h, :n] = s["scores"][b, h, old].double()
            scores[b, h, n:x] = 0.0
    return caches[0], caches[1], scores, _gpu(np.array(lengths, np.int32)), _gpu(index)
