"""attention_weights against its 64-bit form (needs a GB300)."""
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


def _case(dtype, lengths, counts, Hq, Hkv, dim, page, tree=0, seed=0, extra=0, heads_first=False):
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    k, _, pages = refs.paged(DT[dtype], [a + n for a, n in zip(lengths, counts)], Hkv, dim, page, seed, heads_first)
    T = sum(counts) + extra
    q = torch.randn((T, Hq, dim), generator=g).to(DT[dtype])
    starts = np.cumsum([0] + list(counts)).astype(np.int32)
    mask = np.stack([random_tree(tree, max(1, tree // 6), rng)[2] for _ in lengths]) if tree else None
    # the rows' sums: close to what attention over the same positions gives, so that weights are of their usual size
    lse = torch.tensor([[math.log(max(1, a + n)) + 0.5 for a, n in zip(lengths, counts) for _ in range(n)] +
                        [0.0] * extra], dtype=torch.float32).T.repeat(1, Hq) + torch.rand((T, Hq), generator=g)
    return dict(q=q, k=k, pages=pages, starts=starts, mask=mask, lse=lse.contiguous(), lengths=lengths, counts=counts,
                heads_first=heads_first)


def _run(D, s, scores, scale=None, err=None):
    k = s["k"].cuda()
    k = k.transpose(1, 2) if s["heads_first"] else k
    q = s["q"].cuda() if s["q"].is_contiguous() else s["q"][:1].cuda().expand(s["q"].shape)
    return D.attention_weights(q, k, s["pages"].cuda(), _i32(s["lengths"]), _i32(s["starts"]),
                               s["lse"].cuda(), scores, scale=scale, device_err=err,
                               mask=None if s["mask"] is None else torch.from_numpy(s["mask"]).cuda())


def _check(D, s, scale=None, extra_width=7):
    k = s["k"].transpose(1, 2) if s["heads_first"] else s["k"]
    Hkv, dim = k.shape[2], k.shape[3]
    B = len(s["lengths"])
    width = max(a + n for a, n in zip(s["lengths"], s["counts"])) + extra_width
    g = torch.Generator().manual_seed(1)
    before = torch.rand((B, Hkv, width), generator=g)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scores = before.cuda()
    got = _run(D, s, scores, scale, err)
    assert got.data_ptr() == scores.data_ptr() and err.item() == 0
    got = got.cpu()
    for b, (a, n) in enumerate(zip(s["lengths"], s["counts"])):
        S = a + n if n else 0
        rows = slice(s["starts"][b], s["starts"][b] + n)
        key = refs.rows_of(k, s["pages"], b, S)
        total, bound = refs.weights(s["q"][rows], key, s["lse"][rows], dim ** -0.5 if scale is None else scale, a, n,
                                    None if s["mask"] is None else s["mask"][b])
        want = before[b, :, :S].double().numpy() + total
        # one rounding of the sum to fp32
        slack = bound + refs.U * np.abs(want)
        off = np.abs(got[b, :, :S].double().numpy() - want)
        assert np.all(off <= slack), (b, float((off / slack).max()))
        assert torch.equal(got[b, :, S:], before[b, :, S:])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,dim", [(32, 8, 128), (8, 8, 64), (7, 1, 128), (3, 1, 8), (6, 2, 72), (71, 1, 64),
                                        (16, 2, 80), (4, 4, 40)])
def test_heads(D, dtype, Hq, Hkv, dim):
    _check(D, _case(dtype, [0, 130, 517, 64], [1, 1, 1, 1], Hq, Hkv, dim, 16, seed=Hq))
    _check(D, _case(dtype, [0, 129, 1, 255], [5, 70, 129, 1], Hq, Hkv, dim, 32, seed=Hq + 1))


@pytest.mark.parametrize("page", [8, 16, 24, 64, 128, 256])
@pytest.mark.parametrize("heads_first", [False, True])
def test_pages(D, page, heads_first):
    _check(D, _case("bf16", [300, 0, 127, 128, 1], [3, 2, 1, 1, 4], 8, 2, 64, page, seed=page, heads_first=heads_first))


@pytest.mark.parametrize("tree,lead,lengths", [(5, 1, [100, 0, 126]), (78, 1, [300, 127, 50]), (100, 3, [0, 200, 60]),
                                               (496, 1, [40, 700]), (33, 0, [95, 128, 0]), (1024, 1, [31])])
def test_trees(D, tree, lead, lengths):
    _check(D, _case("bf16", lengths, [tree + lead] * len(lengths), 8, 2, 128, 16, tree=tree, seed=tree))


def test_chunks_shorter_than_the_tree(D):
    _check(D, _case("f16", [100, 20, 64, 7], [21, 4, 1, 0], 4, 2, 64, 16, tree=20, seed=2))


@pytest.mark.parametrize("n", [60, 257, 600])
def test_many_row_blocks(D, n):
    """Chunks of one, two, three and more blocks of rows in one call, and sequences without a chunk."""
    _check(D, _case("bf16", [0, 500, 90, 1000, 3], [n, 1, 0, n // 2, n], 16, 2, 64, 64, seed=n, extra=3))


@pytest.mark.parametrize("Hq,Hkv,n", [(300, 1, 3), (512, 1, 2), (514, 2, 4), (256, 1, 5)])
def test_more_queries_than_a_block_has_rows(D, Hq, Hkv, n):
    _check(D, _case("bf16", [200, 0, 130], [n, 1, n], Hq, Hkv, 64, 16, seed=Hq, extra=1))
    _check(D, _case("f16", [90], [34], Hq, Hkv, 16, 16, tree=33, seed=n))


def test_queries_with_strides(D):
    """Queries that are a part of a projection's output."""
    s = _case("bf16", [100, 300], [5, 1], 6, 2, 64, 16, seed=21)
    want = _run(D, s, torch.zeros((2, 2, 310), device="cuda"))
    wide = torch.randn(6, 10, 64).to(torch.bfloat16)
    wide[:, 2:8] = s["q"]
    got = torch.zeros((2, 2, 310), device="cuda")
    D.attention_weights(wide.cuda()[:, 2:8], s["k"].cuda(), s["pages"].cuda(), _i32(s["lengths"]), _i32(s["starts"]),
                        s["lse"].cuda(), got)
    assert torch.equal(got, want)


def test_many_tiles_a_head(D):
    _check(D, _case("bf16", [20000, 9000], [1, 1], 4, 1, 128, 128, seed=1))
    _check(D, _case("f16", [5000], [300], 8, 2, 128, 64, seed=2))


def test_many_sequences(D):
    _check(D, _case("f16", [(37 * b) % 300 for b in range(500)], [1 + b % 3 for b in range(500)], 4, 2, 32, 16, seed=4))


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0])
def test_scales(D, scale):
    s = _case("bf16", [90], [10], 4, 2, 16, 8, seed=6)
    s["lse"] += 8.0
    _check(D, s, scale=scale)


def test_rows_that_add_nothing(D):
    s = _case("bf16", [200, 50], [40, 1], 8, 2, 64, 16, seed=7)
    s["lse"][3] = math.inf
    s["lse"][5:9] = -math.inf
    s["lse"][11, 2] = math.nan
    s["q"][11, 2] = math.nan
    s["lse"][40] = math.inf                   # the whole of the second chunk
    _check(D, s)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_what_a_row_does_not_see_does_not_reach_it(D, dtype):
    """Infinities and NaN in rows behind the end, in later tokens and in other branches' nodes: a score is made of its
    own position's key alone, and an infinite key reaches no row that is left out."""
    tree = 30
    s = _case(dtype, [100, 37], [tree + 1, tree + 1], 4, 2, 64, 16, tree=tree, seed=8)
    clean = _check(D, s)
    page = 16
    odd = s["k"].clone()
    for b, a in enumerate(s["lengths"]):
        p = torch.tensor([a + 5, a + 9])
        odd[s["pages"][b, p // page].long(), p % page] = torch.tensor([math.nan, math.inf], dtype=odd.dtype)[:, None, None]
        behind = a + tree + 1
        last = s["pages"][b, behind // page]
        if last >= 0:
            odd[last, behind % page:] = math.nan
    s["k"] = odd
    scores = torch.rand((2, 2, 138), generator=torch.Generator().manual_seed(1)).cuda()
    got = _run(D, s, scores).cpu()
    for b, a in enumerate(s["lengths"]):
        keep = torch.ones(138, dtype=torch.bool)
        keep[[a + 5, a + 9]] = False
        assert torch.equal(got[b][:, keep], clean[b][:, keep])
    # a row left out does not take up the infinity either
    s["lse"][:] = math.inf
    scores = torch.zeros((2, 2, 138), device="cuda")
    assert not _run(D, s, scores).any()


def test_with_the_attention_it_follows(D):
    """With the sums that tree_attention returns, each query head's weights add up to one a row."""
    tree = 40
    s = _case("bf16", [700, 129, 0], [tree + 1] * 3, 8, 2, 128, 16, tree=tree, seed=9, extra=2)
    q, k, pages = s["q"].cuda(), s["k"].cuda(), s["pages"].cuda()
    lengths, starts, mask = _i32(s["lengths"]), _i32(s["starts"]), torch.from_numpy(s["mask"]).cuda()
    att = D.tree_attention(q, k, k, pages, lengths, starts, mask=mask, lse=True)
    scores = torch.zeros((3, 2, 750), device="cuda")
    D.attention_weights(q, k, pages, lengths, starts, att["lse"], scores, mask=mask)
    # 41 rows of 4 queries, each row's weights off by 2^-10 at most: its sum was made with the same products
    assert torch.allclose(scores.sum(-1), torch.full((3, 2), 4.0 * (tree + 1), device="cuda"), rtol=2.0 ** -10, atol=0)
    again = torch.zeros((3, 2, 750), device="cuda")
    D.attention_weights(q, k, pages, lengths, starts, att["lse"], again, mask=mask)
    assert torch.equal(again, scores)


def test_out_of_range(D):
    s = _case("bf16", [100, 40], [1, 1], 4, 2, 64, 16, seed=10)
    clean = _run(D, s, torch.zeros((2, 2, 101), device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    short = _run(D, s, torch.zeros((2, 2, 70), device="cuda"), err=err)       # scores for 70 positions
    assert err.item() == 32 and torch.equal(short, clean[..., :70])
    s["pages"][1, 1] = 5000                                                   # reads as zeros
    err.zero_()
    got = _run(D, s, torch.zeros((2, 2, 101), device="cuda"), err=err)
    assert err.item() == 32 and torch.equal(got[0], clean[0])
    zero = torch.exp(-s["lse"][1].view(2, 2)).sum(-1).cuda()
    assert torch.allclose(got[1, :, 16:32], zero[:, None].expand(2, 16), rtol=2.0 ** -20)
    assert torch.equal(got[1, :, :16], clean[1, :, :16])


def test_strided_scores_stream_and_graph(D):
    s = _case("f16", [200, 60], [3, 1], 4, 2, 64, 16, seed=11)
    big = torch.zeros((2, 5, 300), device="cuda")
    part = big[:, 1:5:2, 9:]
    plain = _run(D, s, torch.zeros((2, 2, 291), device="cuda"))
    _run(D, s, part)
    assert torch.equal(part, plain) and not big[:, ::2].any() and not big[:, :, :9].any()
    k, q, pages = s["k"].cuda(), s["q"].cuda(), s["pages"].cuda()
    lengths, starts, lse = _i32(s["lengths"]), _i32(s["starts"]), s["lse"].cuda()
    scores = torch.zeros((2, 2, 291), device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    D.attention_weights(q, k, pages, lengths, starts, lse, scores, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(scores, plain)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.attention_weights(q, k, pages, lengths, starts, lse, scores)
    lengths.copy_(_i32([150, 60]))
    scores.zero_()
    g.replay()
    s["lengths"] = [150, 60]
    assert torch.equal(scores, _run(D, s, torch.zeros((2, 2, 291), device="cuda")))


def test_a_wait_that_runs_out(D):
    s = _case("bf16", [3000], [1], 4, 2, 128, 16, seed=12)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = _run(D, s, torch.zeros((1, 2, 3001), device="cuda"), err=err)
    assert err.item() == 0
    D.set_wait_limit(1)
    try:
        _run(D, s, torch.zeros((1, 2, 3001), device="cuda"), err=err)
        torch.cuda.synchronize()
        assert err.item() == 1
    finally:
        D.set_wait_limit(0)
    assert torch.equal(_run(D, s, torch.zeros((1, 2, 3001), device="cuda")), want)


def test_refusals(D):
    s = _case("bf16", [60], [2], 4, 2, 64, 16, seed=13)
    ok = torch.zeros((1, 2, 62), device="cuda")
    for bad in (ok[:, :1], ok.double(), ok.cpu(), ok[0], ok[:, :1].expand(1, 2, 62)):
        with pytest.raises(D.DartError):
            _run(D, s, bad)
    for key, bad in (("q", s["q"][:1].expand(2, 4, 64)), ("lse", s["lse"].double()), ("lse", s["lse"][:1]), ("q", s["q"].half()), ("q", s["q"][:, :3])):
        t = dict(s)
        t[key] = bad
        with pytest.raises(D.DartError):
            _run(D, t, ok)
