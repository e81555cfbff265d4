"""tree_accept, kv_keep and kv_evict against plain forms (needs a GB300)."""
import math

import numpy as np
import pytest

from tests import verified_refs as refs
from tests.steps_refs import random_tree

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


# ------------------------------------------------------------------- accept

@pytest.mark.parametrize("B,N,width,vocab", [(1, 1, 1, 2), (5, 7, 3, 3), (3, 78, 10, 4), (9, 496, 32, 3),
                                             (2, 1024, 64, 2), (300, 33, 2, 2)])
def test_accept(D, B, N, width, vocab):
    rng = np.random.default_rng(N)
    parents = np.stack([random_tree(N, width, rng)[0] for _ in range(B)])
    tokens = rng.integers(0, vocab, (B, N)).astype(np.int32)       # few tokens: siblings share theirs
    picks = rng.integers(0, vocab, (B, N + 1)).astype(np.int32)
    for depth in sorted({0, 1, min(3, N), N}):
        out = D.tree_accept(_i32(picks), _i32(tokens), _i32(parents), depth)
        for b in range(B):
            path, toks = refs.accept(picks[b], tokens[b], parents[b], depth)
            pad = [-1] * (depth + 1 - len(path))
            assert out["counts"][b].item() == len(path)
            assert out["path"][b].tolist() == path + pad
            assert out["tokens"][b].tolist() == toks + pad


def test_accept_what_cannot_be(D):
    """Parents that are not below their node, negative tokens and picks, a tree without nodes."""
    parents, tokens = [[0, 1, -1, 2, -2, 9]], [[5, 5, 5, -1, 5, 5]]
    picks = [[5, 5, 5, -1, 5, 5, 5]]
    out = D.tree_accept(_i32(picks), _i32(tokens), _i32(parents), 6)
    assert out["path"][0].tolist() == [0, 3, -1, -1, -1, -1, -1] and out["counts"].tolist() == [2]
    assert out["tokens"][0].tolist()[:2] == [5, -1]
    out = D.tree_accept(_i32([[4], [7]]), _i32(np.zeros((2, 0))), _i32(np.zeros((2, 0))), 0)
    assert out["path"].tolist() == [[0], [0]] and out["tokens"].tolist() == [[4], [7]]


# --------------------------------------------------------------------- keep

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,dim,page,heads_first", [(8, 128, 16, False), (1, 8, 8, False), (2, 80, 64, True),
                                                        (3, 72, 24, False), (4, 96, 16, True)])
@pytest.mark.parametrize("N", [1, 13, 300])
def test_keep(D, dtype, heads, dim, page, heads_first, N):
    rng = np.random.default_rng(N + dim)
    lengths = [0, 1, 37, 200, 15]
    B = len(lengths)
    k, v, pages = refs.paged(DT[dtype], [x + N + 1 for x in lengths], heads, dim, page, seed=N, heads_first=heads_first)
    width = min(N + 1, 40)
    path, counts = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = int(rng.integers(0, width + 1)) if b else width
        path[b, :n] = np.sort(rng.choice(N + 1, n, replace=False))
        counts[b] = n
    want = [c.transpose(1, 2).clone() if heads_first else c.clone() for c in (k, v)]
    for b, x in enumerate(lengths):
        rows = x + torch.from_numpy(path[b, :counts[b]]).long()
        for c in want:
            old = c[pages[b, rows // page].long(), rows % page].clone()
            new = x + torch.arange(counts[b])
            c[pages[b, new // page].long(), new % page] = old
    kc, vc = k.cuda(), v.cuda()
    ka, va = (kc.transpose(1, 2), vc.transpose(1, 2)) if heads_first else (kc, vc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    wide = torch.full((B, width + 3), 77, dtype=torch.int32, device="cuda")
    wide[:, :width] = _i32(path)
    out = D.kv_keep(ka, va, pages.cuda(), _i32(lengths), wide[:, :width], _i32(counts), device_err=err)
    assert out.tolist() == [x + int(n) for x, n in zip(lengths, counts)]
    assert err.item() == 0
    assert torch.equal(ka.cpu(), want[0]) and torch.equal(va.cpu(), want[1])


def test_keep_leaves_out_what_is_wrong(D):
    page = 8
    k, v, pages = refs.paged(torch.bfloat16, [40] * 6, 2, 16, page, seed=1, width_extra=0)
    pages[5, 1] = 1000                                     # a page id that does not exist
    lengths = [4, -3, 4, 4, 38, 0]
    path = [[0, 5, 6, 9], [0, 1, 2, 3], [0, 5, 3, 9], [0, 1, 2, 3], [0, 1, 2, 3], [1, 9, 17, 18]]
    counts = [4, 4, 4, 5, 4, 4]
    want_k = k.clone()
    for b, i, j in ((0, 1, 5), (0, 2, 6), (0, 3, 9), (2, 1, 5), (2, 3, 9), (5, 0, 1), (5, 2, 17), (5, 3, 18)):
        src, dst = lengths[b] + j, lengths[b] + i
        want_k[pages[b, dst // page], dst % page] = k[pages[b, src // page], src % page]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = k.cuda(), v.cuda()
    out = D.kv_keep(kc, vc, pages.cuda(), _i32(lengths), _i32(path), _i32(counts), device_err=err)
    # 1: a length below 0; 3: more entries than there are; 4: past its pages; 2 and 5: entries that are left out
    assert out.tolist() == [8, -3, 8, 4, 38, 4]
    assert err.item() == 32
    assert torch.equal(kc.cpu(), want_k)


def test_keep_of_values_that_are_the_keys(D):
    """One memory for both moves once."""
    rng = np.random.default_rng(6)
    page, n = 16, 600
    k, _, pages = refs.paged(torch.bfloat16, [900] * 3, 4, 64, page, seed=6)
    path = np.stack([np.sort(rng.choice(n, 300, replace=False)) for _ in range(3)])
    want = k.clone()
    for b in range(3):
        src, dst = 100 + torch.from_numpy(path[b]), 100 + torch.arange(300)
        want[pages[b, dst // page].long(), dst % page] = k[pages[b, src // page].long(), src % page]
    for _ in range(20):
        kc = k.cuda()
        D.kv_keep(kc, kc, pages.cuda(), _i32([100] * 3), _i32(path), _i32([300] * 3))
        assert torch.equal(kc.cpu(), want)


# -------------------------------------------------------------------- evict

def _evict(D, dtype, lengths, heads, dim, page, scores, keep, first, last, seed=0, heads_first=False):
    B = len(lengths)
    k, v, pages = refs.paged(DT[dtype], lengths, heads, dim, page, seed, heads_first=heads_first)
    kc, vc = k.cuda(), v.cuda()
    ka, va = (kc.transpose(1, 2), vc.transpose(1, 2)) if heads_first else (kc, vc)
    want = [c.transpose(1, 2).clone() if heads_first else c.clone() for c in (k, v)]
    new_scores = scores.clone()
    index = np.full((B, heads, keep), -1, np.int32)
    for b, x in enumerate(lengths):
        n = min(x, keep)
        for h in range(heads):
            kept = torch.tensor(refs.evict(scores[b, h].numpy(), x, keep, first, last), dtype=torch.long)
            assert len(kept) == n
            index[b, h, :n] = kept.numpy()
            new = torch.arange(n)
            for c in want:
                old = c[pages[b, kept // page].long(), kept % page, h].clone()
                c[pages[b, new // page].long(), new % page, h] = old
            new_scores[b, h, n:x] = 0
            new_scores[b, h, :n] = scores[b, h, kept]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sc = scores.cuda()
    out = D.kv_evict(ka, va, pages.cuda(), _i32(lengths), sc, keep, first=first, last=last, device_err=err)
    assert err.item() == 0
    assert out["lengths"].tolist() == [min(x, keep) for x in lengths]
    assert np.array_equal(out["index"].cpu().numpy(), index)
    same = lambda a, b: torch.equal(a.view(torch.int32), b.view(torch.int32))
    assert same(sc.cpu(), new_scores)
    assert torch.equal(ka.cpu(), want[0]) and torch.equal(va.cpu(), want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,dim,page,heads_first", [(8, 128, 16, False), (1, 64, 128, False), (2, 80, 8, True),
                                                        (3, 8, 24, False)])
@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 0, 1), (16, 4, 4), (100, 0, 0), (100, 60, 40), (513, 4, 64)])
def test_evict(D, dtype, heads, dim, page, heads_first, keep, first, last):
    lengths = [1200, 0, 1, keep, keep + 1, 777, max(keep - 1, 0)]
    g = torch.Generator().manual_seed(keep)
    scores = torch.rand((len(lengths), heads, 1300), generator=g) ** 8
    _evict(D, dtype, lengths, heads, dim, page, scores, keep, first, last, seed=dim, heads_first=heads_first)


@pytest.mark.parametrize("kind", ["equal", "few", "nan", "infinite", "negative", "zeros"])
def test_evict_unusual_scores(D, kind):
    g = torch.Generator().manual_seed(3)
    s = torch.rand((2, 2, 3000), generator=g)
    if kind == "equal":
        s.fill_(0.5)
    elif kind == "few":
        s = (s * 4).floor()
    elif kind == "nan":
        s[s < 0.7] = math.nan
    elif kind == "infinite":
        s[s < 0.2] = -math.inf
        s[s > 0.9] = math.inf
    elif kind == "negative":
        s = s - 0.5
    else:
        s = torch.where(s < 0.5, 0.0, -0.0)
    _evict(D, "bf16", [3000, 2500], 2, 16, 8, s, 1100, 3, 10)


# one CTA a head and clusters of them, either number of scores a thread, and more than the registers of eight hold
@pytest.mark.parametrize("B,heads,keep,length", [(1, 1, 20000, 40000), (1, 8, 4096, 9001), (40, 4, 300, 1000),
                                                 (1, 2, 50000, 100001), (1, 1, 1000, 163840), (1, 1, 70000, 163900),
                                                 (100, 2, 5000, 10235), (40, 8, 700, 10300)])
def test_evict_sizes(D, B, heads, keep, length):
    g = torch.Generator().manual_seed(keep)
    _evict(D, "f16", [length - 3 * b for b in range(B)], heads, 32, 64,
           torch.rand((B, heads, length + 5), generator=g), keep, 4, 32)


def test_evict_of_scores_with_strides(D):
    """Scores that are a part of a larger tensor: what lies around them stays."""
    k, v, pages = refs.paged(torch.bfloat16, [100, 90], 2, 16, 8, seed=1)
    g = torch.Generator().manual_seed(1)
    big = torch.rand((2, 3, 130), generator=g).cuda()
    part = big[:, 1:, 4:112]
    before, plain = big.clone(), part.contiguous()
    a = D.kv_evict(k.cuda(), v.cuda(), pages.cuda(), _i32([100, 90]), plain, 30, first=2, last=5)
    b = D.kv_evict(k.cuda(), v.cuda(), pages.cuda(), _i32([100, 90]), part, 30, first=2, last=5)
    assert torch.equal(a["index"], b["index"]) and torch.equal(part, plain)
    before[:, 1:, 4:112] = plain
    assert torch.equal(big, before)


def test_evict_of_values_that_are_the_keys(D):
    lengths, keep, page = [3000, 100, 2500], 1000, 16
    k, _, pages = refs.paged(torch.float16, lengths, 2, 128, page, seed=7)
    scores = torch.rand((3, 2, 3000), generator=torch.Generator().manual_seed(7))
    want = k.clone()
    for b, x in enumerate(lengths):
        for h in range(2):
            kept = torch.tensor(refs.evict(scores[b, h].numpy(), x, keep, 4, 8), dtype=torch.long)
            new = torch.arange(len(kept))
            want[pages[b, new // page].long(), new % page, h] = k[pages[b, kept // page].long(), kept % page, h]
    for _ in range(20):
        kc = k.cuda()
        D.kv_evict(kc, kc, pages.cuda(), _i32(lengths), scores.cuda(), keep, first=4, last=8)
        assert torch.equal(kc.cpu(), want)


def test_evict_lengths_out_of_range(D):
    k, v, pages = refs.paged(torch.bfloat16, [64, 64, 64], 2, 16, 8, seed=1, width_extra=0)
    kc, vc = k.cuda(), v.cuda()
    s = torch.rand((3, 2, 60), device="cuda")
    before = s.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = D.kv_evict(kc, vc, pages.cuda(), _i32([65, -1, 61]), s, 10, device_err=err)
    assert err.item() == 32 and out["lengths"].tolist() == [65, -1, 61]
    assert torch.equal(s, before) and torch.equal(kc.cpu(), k) and bool((out["index"] == -1).all())


def test_refusals(D):
    k, v, pages = refs.paged(torch.bfloat16, [64], 2, 16, 8, seed=1)
    k, v, pages, n = k.cuda(), v.cuda(), pages.cuda(), _i32([50])
    s = torch.zeros((1, 2, 64), device="cuda")
    for kw in (dict(keep=0), dict(keep=5, first=3, last=3), dict(keep=5, first=-1)):
        with pytest.raises(D.DartError):
            D.kv_evict(k, v, pages, n, s, **kw)
    for bad in (s[:, :1], s.double(), s[0], s.cpu(), s.expand(1, 2, 64)[:, :, ::2], s[:, :1].expand(1, 2, 64)):
        with pytest.raises(D.DartError):
            D.kv_evict(k, v, pages, n, bad, 10)
    path = _i32([[0, 1]])
    for bad in (path[:, :0], path.long(), path[0], path.cpu()):
        with pytest.raises(D.DartError):
            D.kv_keep(k, v, pages, n, bad, n)
    t = _i32([[1, 2]])
    for args in ((t, t, t, 1), (_i32([[1, 2, 3]]), t, t, 3), (_i32([[1, 2, 3]]), t, t, -1), (_i32([[1, 2, 3]]), t, t[0], 1)):
        with pytest.raises(D.DartError):
            D.tree_accept(*args)
