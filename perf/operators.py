"""The operators around the draft tree, as timed and compared work.

adjust:  penalties, biases and grammar masks on logits (before a tree is built, and on a verified tree's rows)
append:  norms and rotary positions of queries and keys, keys and values written to a paged cache
attend:  attention of a chunk of new tokens (a causal lead, then a tree with packed ancestor masks) over that cache

``own = False`` computes them in plain 32-bit torch operations, ``own = True`` through the package.  A case is a
dict of plain values; its sequences' lengths follow from those values alone, the numbers in them from the seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _adjust(name=None, **over):
    c = dict(op="adjust", dtype="bf16", B=1, R=8, V=151936, pad=0, history=256, bias=0, tree=0,
             grammar="none", allowed=1.0)
    c.update(over)
    return dict(c, name=name) if name else c


def _append(name=None, **over):
    c = dict(op="append", dtype="bf16", B=1, n=1, ctx=1024, Hq=32, Hkv=8, D=128, rot=128, interleaved=False,
             norm=True, page=64, tree=0, factor=1.0)
    c.update(over)
    return dict(c, name=name) if name else c


def _attend(name=None, **over):
    c = dict(op="attend", dtype="bf16", B=1, n=1, ctx=1024, Hq=32, Hkv=8, D=128, page=64, tree=0)
    c.update(over)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence's eight draft rows in a chat: penalties over the text so far, nothing else
        _adjust("adjust_one_draft", B=1, R=8, history=300),
        # a batch of 64 drafts with penalties over up to 2048 tokens and 300 biased tokens each
        _adjust("adjust_batch_bias", B=64, R=8, history=2048, bias=300),
        # 256 drafts under a grammar with its own mask per row that leaves a few tokens
        _adjust("adjust_grammar_rows", dtype="f16", B=256, R=8, V=32000, history=512, grammar="row", allowed=0.02),
        # the verified rows of four trees (root and 496 nodes): each row's path counts as history; one mask a sequence
        _adjust("adjust_tree_rows", B=4, R=497, tree=496, history=4096, grammar="sequence", allowed=0.9),
        # one token of one sequence
        _append("append_one_token", B=1, n=1, ctx=4097),
        # 64 trees of 78 nodes behind their roots, in 16-token pages
        _append("append_trees", B=64, n=79, ctx=2048, tree=78, page=16),
        # an 8191-token piece of a prompt far into a long context, half of each head rotated, scaled frequencies
        _append("append_prompt", dtype="f16", B=1, n=8191, ctx=120000, rot=64, interleaved=True, norm=False, factor=4.0),
        # one token of one sequence: a decode step's latency
        _attend("attend_one_token", B=1, n=1, ctx=4097),
        # a decode step of 64 sequences of about 6000 tokens: the cache is read once
        _attend("attend_decode_batch", B=64, n=1, ctx=8192),
        # 64 trees of 78 nodes behind their roots over about 1500 tokens each
        _attend("attend_trees", B=64, n=79, ctx=2048, tree=78, page=16),
        # 32 trees of 496 nodes behind their roots over about 3000 tokens each
        _attend("attend_wide_trees", B=32, n=497, ctx=4096, tree=496),
        # the next 2048 tokens of two prompts of up to 32768 tokens: plain causal
        _attend("attend_prompt", dtype="f16", B=2, n=2048, ctx=32768, page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    worst = {}
    for c in listed():
        w = work(c)
        seen = worst.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for key in seen:
            seen[key] = max(seen[key], w[key])
    op = rng.choice(["adjust", "append", "attend"])
    while True:
        if op == "adjust":
            tree = rng.choice([0, 0, _log_int(rng, 5, 496)])
            grammar = rng.choice(["none", "sequence", "row"])
            c = _adjust(dtype=rng.choice(["bf16", "f16", "f32"]), B=_log_int(rng, 1, 256),
                        R=tree + rng.randint(0, 1) if tree else rng.randint(1, 16),
                        V=rng.choice([32000, 151936, _log_int(rng, 1000, 160000)]), pad=rng.choice([0, 0, 8, 61]),
                        history=_log_int(rng, 16, 16384), bias=rng.choice([0, 0, rng.randint(1, 300)]), tree=tree,
                        grammar=grammar, allowed=rng.choice([0.01, 0.2, 0.9]) if grammar != "none" else 1.0)
        else:
            Hkv = rng.choice([1, 2, 4, 8])
            D = rng.choice([64, 96, 128, 128])
            tree = rng.choice([0, 0, _log_int(rng, 5, 496)])
            n = tree + 1 if tree else rng.choice([1, 1, _log_int(rng, 2, 4096)])
            common = dict(dtype=rng.choice(["bf16", "f16"]), B=_log_int(rng, 1, 128), n=n, Hkv=Hkv,
                          Hq=Hkv * rng.choice([1, 3, 4, 7, 8]), D=D, tree=tree, page=rng.choice([16, 32, 64, 128]),
                          ctx=_log_int(rng, 32, 32768))
            if op == "append":
                c = _append(rot=rng.choice([D, D // 2]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.5,
                            factor=rng.choice([1.0, 8.0]), **common)
            else:
                c = _attend(**common)
        w = work(c)
        # the caches are held several times over while cases are compared: keep them below 16 GB
        cache = 4 * c["B"] * (c["ctx"] + c["n"]) * c["Hkv"] * c["D"] if op != "adjust" else 0
        if all(w[key] <= worst[op][key] for key in w) and cache < 16e9:
            return c


def _context(c):
    """Each sequence's tokens before the chunk: the first has all of ctx, the others down to half of it."""
    return [c["ctx"] - (b * 7919) % (c["ctx"] // 2 + 1) for b in range(c["B"])]


def _chunks(c):
    """Each sequence's new tokens: all n of a tree and of a single sequence, else down to half of n."""
    if c["tree"] or c["n"] == 1:
        return [c["n"]] * c["B"]
    return [c["n"] - (b * 104729) % (c["n"] // 2 + 1) for b in range(c["B"])]


def _history(c):
    return [c["history"] - (b * 7919) % (c["history"] // 2 + 1) for b in range(c["B"])]


def work(case):
    c = case
    es = BYTES[c["dtype"]]
    if c["op"] == "adjust":
        logits = c["B"] * c["R"] * c["V"]
        read = logits * es * c["allowed"]          # a banned token's logit need not be read
        masks = {"none": 0, "sequence": c["B"], "row": c["B"] * c["R"]}[c["grammar"]] * 4 * ((c["V"] + 31) // 32)
        small = 4 * sum(_history(c)) + 8 * c["B"] * c["bias"] + c["B"] * c["tree"] * (4 + 4 * ((c["tree"] + 31) // 32))
        return {"bytes": int(read + logits * es + masks + small), "flops": int(4 * logits * c["allowed"])}
    tokens = sum(_chunks(c))
    q, kv = tokens * c["Hq"] * c["D"], tokens * c["Hkv"] * c["D"]
    if c["op"] == "append":
        return {"bytes": es * (2 * q + 4 * kv), "flops": 7 * (q + kv)}
    rows = sum(x + n for x, n in zip(_context(c), _chunks(c)))
    pairs = 0
    for x, n in zip(_context(c), _chunks(c)):
        lead = n - c["tree"]
        pairs += lead * x + lead * (lead + 1) // 2
        # a node sees the context, the lead and its path; paths are counted at the mean depth of the trees made below
        pairs += c["tree"] * (x + lead) + sum(_depths(c["tree"]))
    return {"bytes": es * (2 * q + 2 * rows * c["Hkv"] * c["D"]), "flops": 4 * c["D"] * c["Hq"] * pairs}


# ------------------------------------------------------------------- trees

def _depths(N):
    """Depths of a tree of N nodes as the builder numbers them: depth by depth, at most N // 16 + 4 wide."""
    width, out, depth = N // 16 + 4, [], 1
    while len(out) < N:
        out += [depth] * min(width, N - len(out))
        depth += 1
    return out


def _trees(N, B, rng):
    """parents [B, N] and packed ancestor-or-self masks [B, N, ceil(N / 32)] of random trees with those depths."""
    depth = np.array(_depths(N))
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


# ------------------------------------------------------------------ inputs

def _gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def prepare(case, seed):
    c = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dt)

    s = {"case": c}
    B = c["B"]
    if c["tree"]:
        s["parents"], mask = _trees(c["tree"], B, rng)
        s["mask"] = _gpu(mask)
    if c["op"] == "adjust":
        R, V = c["R"], c["V"]
        s["logits"] = normal(B, R, V + c["pad"], scale=3.0)[..., :V]
        # token use falls off as 1 / rank; the padding behind each history holds -1
        rank = np.exp(rng.uniform(0.0, math.log(V), size=(B, c["history"]))).astype(np.int64) % V
        lens = np.array(_history(c), np.int32)
        rank[np.arange(c["history"])[None, :] >= lens[:, None]] = -1
        s["history"], s["lengths"] = _gpu(rank.astype(np.int32)), _gpu(lens)
        s["repetition"] = _gpu(rng.uniform(1.0, 1.5, B).astype(np.float32))
        s["presence"] = _gpu(rng.uniform(0.0, 1.0, B).astype(np.float32))
        s["frequency"] = _gpu(rng.uniform(0.0, 0.5, B).astype(np.float32))
        if c["bias"]:
            s["bias_ids"] = _gpu(rng.integers(0, V, size=(B, c["bias"])).astype(np.int32))
            s["bias_vals"] = _gpu(rng.uniform(-5.0, 5.0, size=(B, c["bias"])).astype(np.float32))
        if c["tree"]:
            s["tokens"] = _gpu((np.exp(rng.uniform(0.0, math.log(V), size=(B, c["tree"]))).astype(np.int64) % V)
                               .astype(np.int32))
        if c["grammar"] != "none":
            rows, words = (R if c["grammar"] == "row" else 1), (V + 31) // 32
            bits = torch.rand((B, rows, words * 32), generator=gen, device="cuda") < c["allowed"]
            weights = (1 << torch.arange(32, device="cuda", dtype=torch.int64))
            packed = torch.empty((B, rows, words), dtype=torch.int32, device="cuda")
            for b in range(B):
                w = (bits[b].view(rows, words, 32) * weights).sum(-1)
                packed[b] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
            s["allowed"] = packed if c["grammar"] == "row" else packed[:, 0].contiguous()
        return s
    ctx, new = _context(c), _chunks(c)
    P, D, Hq, Hkv = c["page"], c["D"], c["Hq"], c["Hkv"]
    need = [(x + n + P - 1) // P for x, n in zip(ctx, new)]
    total = sum(need) + 3                       # pages in random order, a few of them nobody's
    order = rng.permutation(total)
    table, at = np.zeros((B, max(need)), np.int32), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(starts[-1])
    s.update(ctx=ctx, new=new, pages=_gpu(table), lengths=_gpu(np.array(ctx, np.int32)), starts=_gpu(starts))
    s["k_cache"], s["v_cache"] = normal(total, P, Hkv, D), normal(total, P, Hkv, D)
    if c["op"] == "attend":
        s["q"] = normal(T, Hq, D)
        if own:
            import draft_tree_construction_gb300 as dart
            s["workspace"] = torch.zeros(dart.attention_workspace_bytes(T, B, Hq, Hkv, D), dtype=torch.uint8,
                                         device="cuda")
        return s
    # q, k and v are views of one projection's output
    qkv = normal(T, Hq + 2 * Hkv, D)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if c["tree"]:
        lead = c["n"] - c["tree"]
        offsets = list(range(lead)) + [lead - 1 + d for d in _depths(c["tree"])]
        s["offsets"] = _gpu(np.tile(np.array(offsets, np.int32), B))
    if c["norm"]:
        s["q_weight"] = (1.0 + 0.1 * normal(D).float()).to(dt)
        s["k_weight"] = (1.0 + 0.1 * normal(D).float()).to(dt)
    s["freqs"], s["magnitude"] = _frequencies(c)
    if own:
        import draft_tree_construction_gb300 as dart
        s["rotary"] = dart.Rotary(s["freqs"], magnitude=s["magnitude"], interleaved=c["interleaved"])
    return s


def _frequencies(c):
    """rot / 2 angles per position: 10000^(-2j / rot); stretched by `factor` where a turn takes longer than 2048 / 1
    positions, untouched where it takes less than 2048 / 32, blended in between."""
    half = c["rot"] // 2
    f = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    if c["factor"] == 1.0:
        return f, 1.0
    turns = 2048.0 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return f * keep + f / c["factor"] * (1.0 - keep), 0.1 * math.log(c["factor"]) + 1.0


# ------------------------------------------------------------------- calls

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return {"adjust": _own_adjust, "append": _own_append, "attend": _own_attend}[op](s)
    return {"adjust": _plain_adjust, "append": _plain_append, "attend": _plain_attend}[op](s)


def _own_adjust(s):
    import draft_tree_construction_gb300 as dart
    bias = (s["bias_ids"], s["bias_vals"]) if "bias_ids" in s else None
    return dart.adjust_logits(s["logits"], history=s["history"], lengths=s["lengths"], repetition=s["repetition"],
                              presence=s["presence"], frequency=s["frequency"], bias=bias, allowed=s.get("allowed"),
                              tokens=s.get("tokens"), mask=s.get("mask"))


def _own_append(s):
    import draft_tree_construction_gb300 as dart
    q = dart.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"], s["starts"],
                       rotary=s["rotary"], offsets=s.get("offsets"), q_weight=s.get("q_weight"),
                       k_weight=s.get("k_weight"), eps=EPS)
    return q, s["k_cache"], s["v_cache"]


def _own_attend(s):
    import draft_tree_construction_gb300 as dart
    return dart.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"], s["starts"],
                               mask=s.get("mask"), workspace=s["workspace"])["out"]


def _unpack(words, count):
    """int32 [..., W] -> 0 / 1 int32 [..., count], the lowest bit of each word first."""
    shift = torch.arange(32, device=words.device, dtype=torch.int32)
    return ((words.unsqueeze(-1) >> shift) & 1).flatten(-2)[..., :count]


def _plain_adjust(s):
    z, c = s["logits"], s["case"]
    B, R, V = z.shape
    hist = s["history"]
    inside = (torch.arange(hist.shape[1], device="cuda")[None] < s["lengths"][:, None]) & (hist >= 0) & (hist < V)
    count = torch.zeros((B, V), dtype=torch.int32, device="cuda")
    count.scatter_add_(1, torch.where(inside, hist, 0).long(), inside.int())
    count = count[:, None, :].expand(B, R, V)
    if c["tree"]:
        N = c["tree"]
        count = count.clone()
        ids = s["tokens"].long()[:, None, :].expand(B, N, N)
        count[:, R - N:].scatter_add_(2, ids, _unpack(s["mask"], N))
    x = z.float()
    rep, pres, freq = (s[key][:, None, None] for key in ("repetition", "presence", "frequency"))
    x = torch.where(count > 0, torch.where(x > 0, x / rep, x * rep) - pres - freq * count, x)
    if c["bias"]:
        add = torch.zeros((B, V), dtype=torch.float64, device="cuda")
        add.scatter_add_(1, s["bias_ids"].long(), s["bias_vals"].double())
        x = x + add.float()[:, None, :]
    if c["grammar"] != "none":
        bits = _unpack(s["allowed"], V)
        bits = bits if bits.dim() == 3 else bits[:, None, :]
        x = torch.where(bits == 1, x, -math.inf)
    return x.to(z.dtype)


def _plain_append(s):
    c = s["case"]
    T, D = s["q"].shape[0], c["D"]
    token = torch.arange(T, device="cuda")
    seq = (token[:, None] >= s["starts"][None, 1:].long()).sum(1)
    index = token - s["starts"].long()[seq]
    slot = s["lengths"].long()[seq] + index
    position = s["lengths"].long()[seq] + (s["offsets"].long() if "offsets" in s else index)
    angle = position.double()[:, None] * _gpu(s["freqs"])[None, :]
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * s["magnitude"]).float()[:, None, :]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
        rot, rest = x[..., :c["rot"]], x[..., c["rot"]:]
        if c["interleaved"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            new = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = rot.chunk(2, -1)
            new = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([new, rest], -1).to(DTYPES[c["dtype"]])

    page, row = s["pages"].long()[seq, slot // c["page"]], slot % c["page"]
    s["k_cache"][page, row] = turn(s["k"], s.get("k_weight"))
    s["v_cache"][page, row] = s["v"]
    return turn(s["q"], s.get("q_weight")), s["k_cache"], s["v_cache"]


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, D, P, N = c["Hq"], c["Hkv"], c["D"], c["page"], c["tree"]
    G, outs, at = Hq // Hkv, [], 0
    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        S, lead = x + n, n - N
        page = s["pages"][b, :(S + P - 1) // P].long()
        key = s["k_cache"][page].flatten(0, 1)[:S].float()
        val = s["v_cache"][page].flatten(0, 1)[:S].float()
        q = s["q"][at:at + n].float().view(n, Hkv, G, D)
        seen = torch.arange(S, device="cuda")[None, :] <= x + torch.arange(n, device="cuda")[:, None]
        if N:
            seen[lead:, x + lead:] = _unpack(s["mask"][b], N) == 1
        out = torch.empty((n, Hkv, G, D), dtype=torch.float32, device="cuda")
        for h in range(Hkv):
            score = (q[:, h].reshape(n * G, D) @ key[:, h].T).view(n, G, S) * (1.0 / math.sqrt(D))
            score = score.masked_fill_(~seen[:, None, :], -math.inf)
            top = score.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, 0.0, top)
            e = score.sub_(top).exp_()
            out[:, h] = (e.view(n * G, S) @ val[:, h]).view(n, G, D) / e.sum(-1, keepdim=True).clamp_min(1e-38)
        outs.append(out.view(n, Hq, D).to(s["q"].dtype))
        at += n
    return torch.cat(outs)


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    """What run returns, from the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_adjust(s):
    c = s["case"]
    B, R, V = s["logits"].shape
    out = s["logits"].double()
    hist, lens = s["history"].cpu().numpy(), s["lengths"].cpu().numpy()
    for b in range(B):
        rep, pres, freq = (float(s[key][b]) for key in ("repetition", "presence", "frequency"))
        base = np.bincount(hist[b, :lens[b]], minlength=V)
        lead = R - c["tree"]
        counts = [base] * (lead if c["tree"] else 1)
        if c["tree"]:
            toks, paths = s["tokens"][b].cpu().numpy(), {}
            for i in range(c["tree"]):
                p = int(s["parents"][b, i])
                paths[i] = (paths[p] if p >= 0 else []) + [int(toks[i])]
        add = np.zeros(V)
        if c["bias"]:
            np.add.at(add, s["bias_ids"][b].cpu().numpy(), s["bias_vals"][b].cpu().numpy().astype(np.float64))
        add = _gpu(add)
        n = _gpu(base.astype(np.float64))
        for r in range(R):
            m = n
            if c["tree"] and r >= lead:
                path = torch.tensor(paths[r - lead], device="cuda")
                m = n.index_add(0, path, torch.ones(len(path), dtype=torch.float64, device="cuda"))
            x = out[b, r]
            scaled = torch.where(x > 0, x / rep, x * rep)
            out[b, r] = torch.where(m > 0, scaled - pres, x) - freq * m + add
    if c["grammar"] != "none":
        words = s["allowed"] if s["allowed"].dim() == 3 else s["allowed"][:, None]
        v = torch.arange(V, device="cuda")
        for b in range(B):
            bit = (words[b].long()[:, v // 32] >> (v % 32)) & 1
            out[b].masked_fill_((bit == 0).expand(R, V), -math.inf)
    return out


def _exact_append(s):
    c = s["case"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    q = torch.empty(tuple(s["q"].shape), dtype=torch.float64, device="cuda")
    half, at = c["rot"] // 2, 0
    offsets = s["offsets"].cpu().numpy() if "offsets" in s else None
    freqs = np.asarray(s["freqs"])

    def norm(x, w):
        x = x.double()
        if w is None:
            return x
        return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS) * w.double()

    def turn(x, unit):
        # each pair as a complex number, turned by its unit of that position
        x = x.clone()
        lo, hi = (slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["interleaved"] else \
            (slice(0, half), slice(half, c["rot"]))
        z = torch.complex(x[..., lo], x[..., hi]) * unit[:, None, :]
        x[..., lo], x[..., hi] = z.real, z.imag
        return x

    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        rows = slice(at, at + n)
        pos = x + (offsets[rows].astype(np.float64) if offsets is not None else np.arange(n, dtype=np.float64))
        unit = _gpu(s["magnitude"] * np.exp(1j * np.outer(pos, freqs)))
        q[rows] = turn(norm(s["q"][rows], s.get("q_weight")), unit)
        slot = x + np.arange(n)
        page = s["pages"][b].cpu().numpy()[slot // c["page"]]
        where = (_gpu(page.astype(np.int64)), _gpu(slot % c["page"]))
        kc[where] = turn(norm(s["k"][rows], s.get("k_weight")), unit)
        vc[where] = s["v"][rows].double()
        at += n
    return q, kc, vc


def _exact_attend(s):
    c = s["case"]
    if work(c)["flops"] > 1.5e13:               # beyond about 20 seconds of 64-bit products
        return None
    Hq, Hkv, D, P, N = c["Hq"], c["Hkv"], c["D"], c["page"], c["tree"]
    out, at = torch.empty(tuple(s["q"].shape), dtype=torch.float64, device="cuda"), 0
    for b, (x, n) in enumerate(zip(s["ctx"], s["new"])):
        S, lead = x + n, n - N
        slot = torch.arange(S, device="cuda")
        page = s["pages"][b].long()[slot // P]
        hidden = torch.ones((n, S), dtype=torch.bool)
        for i in range(lead):
            hidden[i, :x + i + 1] = False
        for i in range(N):
            hidden[lead + i, :x + lead] = False
            j = i
            while j >= 0:
                hidden[lead + i, x + lead + j] = False
                j = int(s["parents"][b, j])
        hidden = hidden.cuda()
        for g in range(Hq):
            h = g // (Hq // Hkv)
            key, val = s["k_cache"][page, slot % P, h].double(), s["v_cache"][page, slot % P, h].double()
            score = torch.einsum("nd,sd->ns", s["q"][at:at + n, g].double(), key) / math.sqrt(D)
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), dim=-1)
            out[at:at + n, g] = torch.einsum("ns,sd->nd", weight, val)
        at += n
    return out
