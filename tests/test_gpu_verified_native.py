"""The calls behind a verified tree that _steps_native makes against the same calls by the Python binding, their use
together, and what concerns them all (needs a GB300)."""
import threading

import numpy as np
import pytest

from tests import verified_refs as refs
from tests.steps_refs import random_tree

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def _state(seed=0, tree=30):
    """Two sequences behind a tree each: everything that the five calls take."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    lengths = [100, 37]
    k, v, pages = refs.paged(torch.bfloat16, [x + tree + 1 for x in lengths], 2, 64, 16, seed)
    trees = [random_tree(tree, 6, rng) for _ in lengths]
    T = 2 * (tree + 1)
    return dict(logits=(torch.randn(2, tree + 1, 3000, generator=g) * 3).to(torch.bfloat16).cuda(),
                uniforms=torch.rand(2, tree + 1, generator=g).cuda(), temperature=torch.tensor([0.8, 0.0]).cuda(),
                top_k=_i32([40, 0]), top_p=torch.tensor([0.9, 1.0]).cuda(), min_p=torch.tensor([0.0, 0.1]).cuda(),
                tokens=_i32(rng.integers(0, 3000, (2, tree))), parents=_i32(np.stack([t[0] for t in trees])),
                mask=torch.from_numpy(np.stack([t[2] for t in trees])).cuda(), k=k.cuda(), v=v.cuda(),
                pages=pages.cuda(), lengths=_i32(lengths), starts=_i32([0, tree + 1, T]),
                q=torch.randn(T, 8, 64, generator=g).to(torch.bfloat16).cuda(),
                lse=(torch.rand(T, 8, generator=g) + 4).cuda(), scores=torch.rand(2, 2, 140, generator=g).cuda(),
                depth=5)


def _all(D, s, **kw):
    """All five calls, one after the other; their outputs and the tensors that they write."""
    k, v, scores = s["k"].clone(), s["v"].clone(), s["scores"].clone()
    drawn = D.sample_logits(s["logits"], s["uniforms"], temperature=s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"], **kw)
    walked = D.tree_accept(drawn["tokens"], s["tokens"], s["parents"], s["depth"], **kw)
    assert D.attention_weights(s["q"], k, s["pages"], s["lengths"], s["starts"], s["lse"], scores, mask=s["mask"],
                               **kw) is scores
    lengths = D.kv_keep(k, v, s["pages"], s["lengths"], walked["path"], walked["counts"], **kw)
    kept = D.kv_evict(k, v, s["pages"], lengths, scores, 30, first=2, last=8, **kw)
    return [*drawn.values(), *walked.values(), lengths, *kept.values(), k, v, scores]


def test_native_and_binding_alike(D, monkeypatch):
    from draft_tree_construction_gb300 import _steps, _verified
    s = _state()
    native, taken = _verified._native(), []

    class Watch:
        def __getattr__(self, name):
            f = getattr(native, name)

            def g(*args):
                r = f(*args)
                if name != "bind_verified":
                    taken.append((name, r is not None))
                return r
            return g
    monkeypatch.setattr(_steps, "_native", Watch())
    a = _all(D, s)
    assert taken == [(n, True) for n in ("sample", "accept", "weights", "keep", "evict")]
    monkeypatch.setattr(_steps, "_native", _steps._LeaveAll)
    b = _all(D, s)
    for x, y in zip(a, b, strict=True):
        assert x.dtype == y.dtype and torch.equal(x, y)


def test_streams_and_threads(D):
    """Given streams, and two threads at once on streams of their own."""
    states = [_state(seed) for seed in (1, 2)]
    want = [_all(D, s) for s in states]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _all(D, states[0], stream=side)
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    out = _all(D, states[i])
                stream.synchronize()
                assert all(torch.equal(x, y) for x, y in zip(out, want[i], strict=True))
        except BaseException as e:
            errors.append(e)
    # caches are copied on the threads' own streams: the copies on the side stream's are ordered by the synchronize above
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert len(got) == len(want[0])


def test_captured_and_replayed(D):
    s, other = _state(3), _state(4)
    want = [x.clone() for x in _all(D, other)]
    for _ in range(2):
        _all(D, s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _all(D, s)
    for key, x in other.items():
        if torch.is_tensor(x):
            s[key].copy_(x)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, want, strict=True):
        assert torch.equal(x, y)


def test_a_serving_loop(D):
    """A tree built, appended, attended to, drawn from, walked and kept, step after step, against a cache without trees:
    after each step the cache holds the accepted tokens' keys and values in order, as if they had come one by one."""
    B, d, V, Hq, Hkv, dim, page = 3, 3, 500, 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    # a toy target: a token's vectors and the logits that follow it depend on the token alone
    qkv = rnd(V, Hq + 2 * Hkv, dim).to(torch.bfloat16)
    follow = (rnd(V, V) * 2).to(torch.bfloat16)
    W, k = 4, 4
    N = D.num_nodes(d, k, W)
    pages = torch.arange(B * 16, dtype=torch.int32, device="cuda").view(B, 16)
    kc, vc = (torch.zeros((B * 16, page, Hkv, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scores = torch.zeros((B, Hkv, 16 * page), device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, (B + 1) * (N + 1), N + 1, dtype=torch.int32, device="cuda")
    last = torch.tensor([3, 100, 499], dtype=torch.int32, device="cuda")
    texts = [[] for _ in range(B)]
    for step in range(8):
        draft = follow[last.long()][:, None].expand(B, d, V).contiguous() + (rnd(B, d, V) * 0.5).to(torch.bfloat16)
        tree = D.tree_build(draft, 1.0, k, W, 0.0, -10.0)
        chunk = torch.cat([last[:, None], tree["tokens"]], 1)
        x = qkv[chunk.flatten().long()]
        q = D.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, pages, lengths, starts)
        att = D.tree_attention(q, kc, vc, pages, lengths, starts, mask=tree["mask"], lse=True)
        D.attention_weights(q, kc, pages, lengths, starts, att["lse"], scores, mask=tree["mask"])
        u = torch.rand((B, N + 1), generator=g, device="cuda")
        heat = torch.full((B,), 0.5, device="cuda")
        drawn = D.sample_logits(follow[chunk.long()], u, temperature=heat, top_k=_i32([8] * B))
        walk = D.tree_accept(drawn["tokens"], tree["tokens"], tree["parents"], d)
        lengths = D.kv_keep(kc, vc, pages, lengths, walk["path"], walk["counts"])
        for b in range(B):
            n = int(walk["counts"][b])
            rows = walk["path"][b, :n].tolist()
            texts[b] += [int(chunk[b, r]) for r in rows]
            # each token on the path was drawn at the one before it
            assert all(int(drawn["tokens"][b, r]) == t for r, t in zip(rows, walk["tokens"][b, :n].tolist()))
            last[b] = walk["tokens"][b, n - 1]
            assert int(lengths[b]) == len(texts[b])
            where = torch.arange(len(texts[b]))
            rows_k = kc[pages[b].long()].flatten(0, 1)[where]
            rows_v = vc[pages[b].long()].flatten(0, 1)[where]
            text = torch.tensor(texts[b])
            assert torch.equal(rows_k, qkv[text, Hq:Hq + Hkv]) and torch.equal(rows_v, qkv[text, Hq + Hkv:])
    assert D.device_error(att["workspace"]) == 0
    before = [kc.clone(), vc.clone()]
    kept = D.kv_evict(kc, vc, pages, lengths, scores, 6, first=1, last=2)
    for b in range(B):
        n = int(kept["lengths"][b])
        assert n == min(6, len(texts[b]))
        for h in range(Hkv):
            old = kept["index"][b, h, :n].long()
            assert old.tolist() == sorted(set(old.tolist())) and old[0] == 0
            new = torch.arange(n, device="cuda")
            for c, was in zip((kc, vc), before):
                assert torch.equal(c[pages[b].long()].flatten(0, 1)[new, h], was[pages[b].long()].flatten(0, 1)[old, h])
