"""The steps around a tree, run together as a serving loop runs them (needs a GB300).

adjust_logits -> tree_build -> kv_append -> tree_attention -> adjust_logits on
the nodes' rows, the calls captured into one graph too.  What a node computes
must be what a plain decode of its path computes: its tokens one by one, at
consecutive positions, each attending to everything before it.
"""
import math

import numpy as np
import pytest

from tests import steps_refs as refs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


B, DEPTHS, V, K, W, HQ, HKV, DIM, PAGE, CTX = 2, 4, 1000, 4, 5, 4, 2, 64, 16, 45


def _model(seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return dict(embed=r(V, 96), qkv=r(96, (HQ + 2 * HKV) * DIM) / math.sqrt(96), unembed=r(HQ * DIM, V) / 16,
                draft=(r(B, DEPTHS, V) * 3).bfloat16(), q_weight=(1 + 0.1 * r(DIM)).bfloat16(),
                k_weight=(1 + 0.1 * r(DIM)).bfloat16(),
                context=torch.randint(0, V, (B, CTX + 1), generator=g, dtype=torch.int32))


def test_a_verification_step(D):
    m = _model(0)
    cuda = {k: v.cuda() for k, v in m.items()}
    rng = np.random.default_rng(1)
    allowed = rng.integers(0, 2 ** 32, (B, (V + 31) // 32), dtype=np.uint64).astype(np.uint32)
    allow = torch.from_numpy(allowed.view(np.int32)).cuda()
    lens = torch.tensor([CTX + 1, CTX - 6], dtype=torch.int32, device="cuda")     # committed tokens, the root the last
    pages = torch.randperm(12, generator=torch.Generator().manual_seed(2)).int().view(B, 6).cuda()
    caches = [torch.full((12, PAGE, HKV, DIM), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rotary = D.Rotary(D.rotary_frequencies(DIM, factor=4.0, original=64)[0])
    rep = torch.full((B,), 1.3, device="cuda")
    pres = torch.full((B,), 0.2, device="cuda")
    freq = torch.full((B,), 0.1, device="cuda")
    N = D.num_nodes(DEPTHS, K, W)

    def project(tokens):
        return (cuda["embed"][tokens.long()] @ cuda["qkv"]).bfloat16().view(-1, HQ + 2 * HKV, DIM)

    def append(x, lengths, starts, offsets):
        return D.kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], *caches, pages, lengths, starts,
                           rotary=rotary, offsets=offsets, q_weight=cuda["q_weight"], k_weight=cuda["k_weight"])

    # the prompt, without each sequence's last token (the root enters with its tree)
    rows = torch.cat([cuda["context"][b, :int(lens[b]) - 1] for b in range(B)])
    starts0 = torch.tensor([0, int(lens[0]) - 1, int(lens.sum()) - 2], dtype=torch.int32, device="cuda")
    append(project(rows), torch.zeros_like(lens), starts0, None)

    before = lens - 1
    starts = (torch.arange(B + 1, device="cuda") * (N + 1)).int()
    root = torch.stack([cuda["context"][b, int(lens[b]) - 1] for b in range(B)])[:, None]

    def step():
        z = D.adjust_logits(cuda["draft"], history=cuda["context"], lengths=lens, repetition=rep, presence=pres,
                            frequency=freq, allowed=allow)
        tree = D.tree_build(z, 0.8, K, W, 0.0, 0.0)
        chunk = torch.cat([root, tree["tokens"]], 1).reshape(-1)
        offsets = torch.cat([torch.zeros_like(root), tree["pos"]], 1).reshape(-1).contiguous()
        q = append(project(chunk), before, starts, offsets)
        att = D.tree_attention(q, *caches, pages, before, starts, mask=tree["mask"])
        logits = (att["out"].float().view(B, N + 1, -1) @ cuda["unembed"]).bfloat16()
        final = D.adjust_logits(logits, history=cuda["context"], lengths=lens, repetition=rep, presence=pres,
                                frequency=freq, allowed=allow, tokens=tree["tokens"], mask=tree["mask"])
        return tree, q, att, logits, final

    tree, q, att, logits, final = step()
    assert D.device_error(tree["workspace"]) == 0 and D.device_error(att["workspace"]) == 0
    tokens, parents = tree["tokens"].cpu().numpy(), tree["parents"].cpu().numpy()
    bits = refs.unpack(allowed, V)
    assert all(bits[b, tokens[b]].all() for b in range(B))                # the grammar held in the tree

    # attention of every row against the definition, on the cache as it stands
    want, _, bound, _ = refs.attend(q.cpu(), caches[0].cpu(), caches[1].cpu(), pages.cpu().numpy(),
                                    before.cpu().numpy(), starts.cpu().numpy(), tree["mask"].cpu().numpy(),
                                    DIM ** -0.5)
    refs.close(att["out"], want, bound, torch.bfloat16)

    # and against a plain decode of some nodes' paths: the same rows, from a cache of their own
    for b in range(B):
        for node in (0, N // 2, N - 1):
            path, j = [], node
            while j >= 0:
                path.append(j)
                j = int(parents[b, j])
            path = path[::-1]
            seq = [int(t) for t in m["context"][b, :int(lens[b])]] + [int(tokens[b, j]) for j in path]
            alone = [torch.zeros(6, PAGE, HKV, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            table = torch.arange(6, dtype=torch.int32, device="cuda")[None]
            x = project(torch.tensor(seq, device="cuda"))
            zero, all_ = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, len(seq)]).int().cuda()
            qq = D.kv_append(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], *alone, table, zero, all_, rotary=rotary,
                             q_weight=cuda["q_weight"], k_weight=cuda["k_weight"])
            assert torch.equal(qq[-1], q[b * (N + 1) + 1 + node])
            got = D.tree_attention(qq, *alone, table, zero, all_)["out"][-1]
            # both are within their bound of one value
            row = b * (N + 1) + 1 + node
            slack = 2 * (refs.half_step(torch.bfloat16) * (want[row].abs() + bound[row]) + bound[row])
            assert bool(((got.double().cpu() - att["out"][row].double().cpu()).abs() <= slack).all())

    # the adjusted rows, each with its own path
    args = [x.cpu().numpy() for x in (cuda["context"], lens, rep, pres, freq)]
    fw, fb = refs.adjust(logits.cpu(), *args, None, allowed.view(np.int32), tokens, tree["mask"].cpu().numpy())
    refs.close(final, fw, fb, torch.bfloat16)

    # the whole step as one graph: the same bits
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[0]["tokens"], tree["tokens"]) and torch.equal(again[2]["out"], att["out"])
    assert torch.equal(again[4].view(torch.int16), final.view(torch.int16))


@pytest.mark.parametrize("heads_first", [False, True])
def test_pages_whose_offsets_pass_32_bits(D, heads_first):
    """A cache of 2^32 elements and more: the pages at its end serve like those of a small cache, and the tokens
    before the first sequence and behind the last one stay as they were."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    hq, hkv, dim, page, B, width = 8, 4, 128, 64, 3, 5
    count = 2 ** 32 // (page * hkv * dim) + B * width + 1
    shape = (count, hkv, page, dim) if heads_first else (count, page, hkv, dim)
    far = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    near = [torch.zeros((B * width,) + shape[1:], dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    low = torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width)
    high = low + (count - B * width)
    for f, n in zip(far, near):
        n.normal_(generator=gen)
        f[-B * width:] = n
    lengths = torch.tensor([100, 0, 250], dtype=torch.int32, device="cuda")
    starts = torch.tensor([2, 42, 43, 103], dtype=torch.int32, device="cuda")
    qkv = torch.randn(106, hq + 2 * hkv, dim, device="cuda", generator=gen).bfloat16()
    results = []
    for caches, pages in ((near, low), (far, high)):
        view = [c.transpose(1, 2) if heads_first else c for c in caches]
        q = torch.full((106, hq, dim), 3.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        D.kv_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], *view, pages, lengths, starts,
                    rotary=D.Rotary(*D.rotary_frequencies(dim)), out=q, device_err=err)
        att = D.tree_attention(q, *view, pages, lengths, starts, out=torch.full_like(q, 4.0))
        assert int(err) == 0 and D.device_error(att["workspace"]) == 0
        assert bool((q[[0, 1, 103, 104, 105]] == 3).all()) and bool((att["out"][[0, 1, 103, 104, 105]] == 4).all())
        results.append((q, att["out"], caches[0][-B * width:].clone(), caches[1][-B * width:].clone()))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert not torch.equal(results[0][2], torch.zeros_like(results[0][2]))
