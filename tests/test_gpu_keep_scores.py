"""kv_keep with the scores that attention_weights has gathered (needs a GB300)."""
import numpy as np
import pytest

from tests import verified_refs as refs

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


def _case(lengths, chunks, width, heads, dim, page, seed, dtype="bf16"):
    """Caches, pages, paths (every row of which may be shorter), and scores that are nowhere zero."""
    rng = np.random.default_rng(seed)
    B = len(lengths)
    k, v, pages = refs.paged(DT[dtype], [x + n for x, n in zip(lengths, chunks)], heads, dim, page, seed)
    path, counts = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    for b, n in enumerate(chunks):
        counts[b] = min(width, n) if b == 0 else rng.integers(0, min(width, n) + 1)
        path[b, :counts[b]] = np.sort(rng.choice(n, counts[b], replace=False))
    scores = torch.from_numpy(rng.random((B, heads, max(x + n for x, n in zip(lengths, chunks)) + 9)).astype(np.float32) + 1)
    starts = np.concatenate([[3], 3 + np.cumsum(chunks)])
    return k, v, pages, path, counts, scores, starts


def _followed(scores, lengths, chunks, path, counts):
    out = scores.clone()
    for b, (x, n, m) in enumerate(zip(lengths, chunks, counts)):
        out[b, :, x + m:x + n] = 0
        out[b, :, x:x + m] = scores[b][:, x + torch.from_numpy(path[b, :m]).long()]
    return out


# one CTA a head, and clusters of two to eight
@pytest.mark.parametrize("lengths,chunks,width,heads,dim,page",
                         [([0, 1, 37, 200, 15], [1, 7, 14, 301, 40], 40, 8, 128, 16), ([5], [1], 1, 1, 8, 8),
                          ([100], [600], 600, 1, 64, 64), ([31, 0], [2100, 1500], 2100, 1, 16, 32),
                          ([9, 9, 9], [0, 50, 0], 20, 3, 72, 24)])
@pytest.mark.parametrize("same", [False, True])
def test_scores_follow_the_path(D, lengths, chunks, width, heads, dim, page, same):
    k, v, pages, path, counts, scores, starts = _case(lengths, chunks, width, heads, dim, page, seed=width)
    want = _followed(scores, lengths, chunks, path, counts)
    wide = torch.full((len(lengths), heads + 2, scores.shape[2] + 7), 5.0, device="cuda")
    part = wide[:, 1:1 + heads, 4:4 + scores.shape[2]]
    part.copy_(scores.cuda())
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ka, va, kb, vb = k.cuda(), v.cuda(), k.cuda(), v.cuda()
    if same:
        va, vb = ka, kb
    plain = D.kv_keep(kb, vb, pages.cuda(), _i32(lengths), _i32(path), _i32(counts))
    out = D.kv_keep(ka, va, pages.cuda(), _i32(lengths), _i32(path), _i32(counts), scores=part, starts=_i32(starts),
                    device_err=err)
    assert err.item() == 0 and torch.equal(out, plain)
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    assert torch.equal(part.cpu(), want)
    part.fill_(5.0)
    assert bool((wide == 5.0).all())


def test_scores_of_what_is_wrong(D):
    """What the rows of the cache are left out for, the scores are too; and positions that have none."""
    k, v, pages = refs.paged(torch.bfloat16, [40] * 6, 2, 16, 8, seed=1, width_extra=0)
    lengths = [4, -3, 4, 4, 38, 24]
    path = [[0, 5, 6, 9], [0, 1, 2, 3], [0, 5, 3, 9], [0, 1, 2, 3], [0, 1, 2, 3], [0, 5, 7, 8]]
    counts = [4, 4, 4, 5, 4, 4]
    starts = [0, 10, 20, 30, 40, 50, 60]
    s = torch.rand((6, 2, 32), generator=torch.Generator().manual_seed(1)) + 1
    want = s.clone()
    want[0, :, 5:8] = s[0][:, [9, 10, 13]]
    want[0, :, 8:14] = 0
    want[2, :, 5] = s[2, :, 9]                 # 3 behind 5 is left out
    want[2, :, 7] = s[2, :, 13]
    want[2, :, 8:14] = 0
    want[5, :, 25] = s[5, :, 29]               # what lies behind position 31 has no score
    want[5, :, 26] = s[5, :, 31]
    want[5, :, 27:] = 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sc = s.cuda()
    out = D.kv_keep(k.cuda(), v.cuda(), pages.cuda(), _i32(lengths), _i32(path), _i32(counts), scores=sc,
                    starts=_i32(starts), device_err=err)
    assert out.tolist() == [8, -3, 8, 4, 38, 28] and err.item() == 32
    assert torch.equal(sc.cpu(), want)
    # a chunk that reaches behind the scores says so by itself
    err.zero_()
    D.kv_keep(k.cuda(), v.cuda(), pages.cuda(), _i32([24] * 6), _i32([[0]] * 6), _i32([1] * 6), scores=sc,
              starts=_i32(starts), device_err=err)
    assert err.item() == 32 and bool((sc[:, :, 25:] == 0).all())


def test_native_and_binding_alike(D, monkeypatch):
    from draft_tree_construction_gb300 import _steps
    lengths, chunks = [20, 7], [30, 12]
    k, v, pages, path, counts, scores, starts = _case(lengths, chunks, 9, 2, 64, 16, seed=2)
    outs = []
    for native in (_steps._load_native(), _steps._LeaveAll):
        monkeypatch.setattr(_steps, "_native", native)
        ka, va, sc = k.cuda(), v.cuda(), scores.cuda()
        n = D.kv_keep(ka, va, pages.cuda(), _i32(lengths), _i32(path), _i32(counts), scores=sc, starts=_i32(starts))
        outs.append([n, ka, va, sc])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(outs[0][3].cpu(), _followed(scores, lengths, chunks, path, counts))


def test_captured_and_replayed(D):
    """A captured call follows the paths, lengths and starts of the replay."""
    a = _case([20, 7], [30, 12], 9, 2, 64, 16, seed=3)
    b = _case([18, 9], [25, 17], 9, 2, 64, 16, seed=4)
    k, v, pages = a[0].cuda(), a[1].cuda(), a[2].cuda()
    # the width of the scores differs: those of the wider one serve both
    width = max(a[5].shape[2], b[5].shape[2])
    path, counts, starts, lengths = _i32(a[3]), _i32(a[4]), _i32(a[6]), _i32([20, 7])
    sc = torch.ones((2, 2, width), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        D.kv_keep(k, v, pages, lengths, path, counts, scores=sc, starts=starts)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.kv_keep(k, v, pages, lengths, path, counts, scores=sc, starts=starts)
    path.copy_(_i32(b[3])), counts.copy_(_i32(b[4])), starts.copy_(_i32(b[6])), lengths.copy_(_i32([18, 9]))
    s = torch.rand((2, 2, width), generator=torch.Generator().manual_seed(5))
    sc.copy_(s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(sc.cpu(), _followed(s, [18, 9], [25, 17], b[3], b[4]))
