"""tree_attention against its 64-bit form (needs a GB300)."""
import math

import numpy as np
import pytest

from tests import steps_refs as refs

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


def _case(dtype, lengths, counts, Hq, Hkv, dim, page, N=0, heads_first=False, extra=0, seed=0, peaky=1.0):
    """CPU tensors.  Rows of the pages behind each sequence's end hold NaN, unused pages infinities."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, T = len(lengths), sum(counts) + extra
    q = (torch.randn(T, Hq, dim, generator=g) * peaky).to(DT[dtype])
    need = [(a + n + page - 1) // page for a, n in zip(lengths, counts)]
    total, width = sum(need) + 2, max(need) + 2
    order = rng.permutation(total)
    pages, at = np.full((B, width), total - 1, np.int32), 0
    shape = (total, page, Hkv, dim)
    k, v = (torch.randn(shape, generator=g).to(DT[dtype]) for _ in range(2))
    used = torch.zeros(total, page, dtype=torch.bool)
    for b, m in enumerate(need):
        pages[b, :m] = order[at:at + m]
        S = lengths[b] + counts[b]
        for j in range(m):
            used[pages[b, j], :max(0, min(page, S - j * page))] = True
        at += m
    whole = used.any(-1)
    for c in (k, v):
        c[~used] = math.nan
        c[~whole] = math.inf
    mask = None
    if N:
        mask = np.stack([refs.random_tree(N, max(1, N // 5), rng)[2] for _ in range(B)])
    s = dict(q=q, k_cache=k, v_cache=v, pages=pages, lengths=np.array(lengths, np.int32),
             starts=np.cumsum([0] + list(counts)).astype(np.int32), mask=mask, heads_first=heads_first)
    return s


def _cuda(s):
    d = {n: (torch.from_numpy(x).cuda() if isinstance(x, np.ndarray) else x) for n, x in s.items()}
    d["q"] = s["q"].cuda()
    for c in ("k_cache", "v_cache"):
        d[c] = s[c].transpose(1, 2).contiguous().cuda().transpose(1, 2) if s["heads_first"] else s[c].cuda()
    return d


def _args(d):
    return d["q"], d["k_cache"], d["v_cache"], d["pages"], d["lengths"], d["starts"]


def _check(D, s, scale=None, **kw):
    d = _cuda(s)
    T, Hq, dim = s["q"].shape
    out = torch.full((T, Hq, dim), 5.0, dtype=s["q"].dtype, device="cuda")
    got = D.tree_attention(*_args(d), mask=d["mask"], scale=scale, out=out, lse=True, **kw)
    assert D.device_error(got["workspace"]) == 0
    want, lse, bound, lse_bound = refs.attend(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"],
                                              s["starts"], s["mask"], scale if scale is not None else dim ** -0.5)
    inside = ~torch.isnan(want[:, 0, 0])
    refs.close(got["out"][inside.cuda()], want[inside], bound[inside], s["q"].dtype)
    refs.close(got["lse"][inside.cuda()], lse[inside], lse_bound[inside], torch.float32)
    assert bool((got["out"][~inside.cuda()] == 5.0).all())                # rows of no sequence stay
    return d, got


CASES = [
    # dtype, lengths, counts, Hq, Hkv, dim, page, N, heads first, rows behind
    ("bf16", [700], [1], 8, 2, 128, 64, 0, False, 0),
    ("bf16", [0], [1], 1, 1, 128, 16, 0, False, 0),                       # one token, no context
    ("f16", [5, 128, 127, 129, 0], [1, 1, 1, 1, 1], 8, 8, 64, 16, 0, False, 3),
    ("bf16", [300, 0, 60], [33, 40, 0], 8, 2, 128, 32, 32, False, 2),      # trees behind their roots; an empty one
    ("f16", [250, 77], [78, 78], 4, 1, 128, 16, 78, True, 0),              # nodes alone
    ("bf16", [100, 3], [50, 20], 6, 2, 96, 24, 40, False, 0),              # a chunk shorter than its tree
    ("bf16", [130], [257], 2, 1, 128, 128, 0, True, 0),                    # a prompt's piece, causal
    ("f16", [0, 0], [140, 300], 7, 1, 72, 8, 0, False, 1),
    ("bf16", [1000], [97], 32, 1, 64, 256, 96, False, 0),                  # 32 query heads on one key head
    ("f16", [64, 64], [2, 3], 5, 5, 8, 8, 0, False, 0),
    ("bf16", [2, 5], [200, 129], 3, 1, 128, 40, 129, False, 0),
    ("bf16", [3000] * 3 + [17], [1] * 4, 16, 4, 128, 64, 0, False, 0),
    ("f16", [31] * 40, [5] * 40, 4, 2, 128, 16, 4, False, 0),              # more sequences than lanes
]


@pytest.mark.parametrize("dtype,lengths,counts,Hq,Hkv,dim,page,N,heads_first,extra", CASES)
def test_attention_matches_the_definition(D, dtype, lengths, counts, Hq, Hkv, dim, page, N, heads_first, extra):
    s = _case(dtype, lengths, counts, Hq, Hkv, dim, page, N, heads_first, extra, seed=Hq + page)
    _check(D, s)


@pytest.mark.parametrize("scale,peaky", [(0.0, 1.0), (-0.3, 1.0), (1.0, 4.0)])
def test_scales_and_peaks(D, scale, peaky):
    """Uniform weights, a negative scale, and scores hundreds apart."""
    _check(D, _case("bf16", [333], [40], 4, 2, 128, 16, 30, seed=3, peaky=peaky), scale=scale)


def test_rows_whose_mask_leaves_nothing(D):
    s = _case("bf16", [0, 40], [20, 20], 4, 2, 64, 16, 20, seed=4)
    s["mask"][0, 3] = 0
    s["mask"][0, 11] = 0
    s["mask"][1, 5] = 0                                                   # still sees its context
    d, got = _check(D, s)
    assert bool((got["out"][3] == 0).all()) and bool((got["lse"][11] == -math.inf).all())


@pytest.mark.parametrize("dtype,lengths,counts,Hq,Hkv,dim,page,N,heads_first", [
    ("bf16", [200, 0, 90], [65, 65, 40], 8, 2, 128, 16, 64, False),       # trees; a chunk of leads and nodes
    ("f16", [70, 5], [150, 129], 4, 1, 64, 32, 0, True),                  # causal: later tokens of the chunk
    ("bf16", [128] * 30, [79] * 30, 32, 8, 72, 24, 78, False),            # blocks of one and of two halves
    ("f16", [5000], [100], 16, 1, 128, 64, 99, False),                    # joined blocks
])
def test_what_a_row_does_not_see_does_not_reach_it(D, dtype, lengths, counts, Hq, Hkv, dim, page, N, heads_first):
    """NaN and infinities in keys and values of positions that some rows see and others do not: the others keep
    the bits they have without them, and the rows that see one of the values' have it in its column."""
    s = _case(dtype, lengths, counts, Hq, Hkv, dim, page, N, heads_first, seed=12)
    rng = np.random.default_rng(12)
    odd = {}                                          # row of q -> {(kv head, column): value}
    keys = torch.zeros(sum(counts), Hkv, dtype=torch.bool)      # rows that see a NaN key
    plain, given = [c.clone() for c in (s["k_cache"], s["v_cache"])], [s["k_cache"], s["v_cache"]]
    for b, (at, n) in enumerate(zip(lengths, counts)):
        lead = max(n - N, 0)
        see = np.stack([refs.visible(at, n, N, i, s["mask"][b, i - lead] if i >= lead else None) for i in range(n)])
        for j, p in enumerate(rng.choice(np.arange(at + 1, at + n), 3, replace=False)):
            h, col = int(rng.integers(Hkv)), int(rng.integers(dim))
            where = (int(s["pages"][b, p // page]), int(p % page), h)
            rows = [int(s["starts"][b]) + i for i in range(n) if see[i, p]]
            if j == 0:                                # a key
                given[0][where + (col,)] = math.nan
                keys[rows, h] = True
            else:
                x = (math.nan, math.inf, -math.inf)[(b + j) % 3]
                given[1][where + (col,)] = x
                plain[1][where + (col,)] = 0.0
                for r in rows:
                    old = odd.setdefault(r, {}).get((h, col), 0.0)
                    odd[r][h, col] = old + x          # inf - inf is NaN
    d = _cuda(s)
    got = D.tree_attention(*_args(d), mask=d["mask"], lse=True)
    assert D.device_error(got["workspace"]) == 0
    d2 = _cuda(dict(s, k_cache=plain[0], v_cache=plain[1]))
    ref = D.tree_attention(*_args(d2), mask=d2["mask"], lse=True)
    want, G = ref["out"].cpu().clone(), Hq // Hkv
    for r, cells in odd.items():
        for (h, col), x in cells.items():
            want[r, h * G:(h + 1) * G, col] = x
    spoilt = keys.repeat_interleave(G, 1)
    out, lse = got["out"].cpu(), got["lse"].cpu()
    assert bool(out[spoilt].isnan().all()) and bool(lse[spoilt].isnan().all())
    assert torch.equal(lse[~spoilt], ref["lse"].cpu()[~spoilt])
    assert torch.equal(out[~spoilt].isnan(), want[~spoilt].isnan())
    assert torch.equal(out[~spoilt].nan_to_num(nan=7.0), want[~spoilt].nan_to_num(nan=7.0))


def test_mask_bits_behind_the_chunk_are_ignored(D):
    s = _case("f16", [10], [25], 2, 1, 64, 8, 25, seed=5)
    d, got = _check(D, s)
    s["mask"][..., 0] |= np.int32(-2 ** 31 + 2 ** 30 + 2 ** 25)           # bits 25, 30, 31
    _, again = _check(D, s)
    assert torch.equal(got["out"], again["out"])


def test_strided_queries_and_a_reused_workspace(D):
    s = _case("bf16", [90, 300], [17, 33], 4, 2, 128, 16, seed=6)
    d = _cuda(s)
    ref = D.tree_attention(*_args(d))["out"]
    wide = torch.zeros(50, 12, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:7] = d["q"]
    room = torch.zeros(50, 8, 136, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(D.attention_workspace_bytes(50, 2, 4, 2, 128), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        D.tree_attention(wide[:, 3:7], *_args(d)[1:], out=room[:, ::2, :128], workspace=ws)
        assert torch.equal(room[:, ::2, :128], ref)
    assert int(room[:, 1::2].abs().max()) == 0 and int(room[:, :, 128:].abs().max()) == 0
    assert D.device_error(ws) == 0


def test_ids_and_lengths_out_of_range_are_reported(D):
    s = _case("bf16", [100, 100], [4, 4], 2, 1, 64, 16, seed=7)
    d = _cuda(s)
    good = D.tree_attention(*_args(d))["out"]
    d["pages"][1, 2] = 10 ** 6
    got = D.tree_attention(*_args(d))
    assert D.device_error(got["workspace"]) == 32
    assert torch.equal(got["out"][:4], good[:4])
    d["pages"][1, 2] = -7
    got = D.tree_attention(*_args(d))
    assert D.device_error(got["workspace"]) == 32 and torch.equal(got["out"][:4], good[:4])
    d = _cuda(s)
    d["lengths"][1] = 10 ** 9                         # far more than its pages hold
    got = D.tree_attention(*_args(d))
    assert D.device_error(got["workspace"]) == 32 and torch.equal(got["out"][:4], good[:4])


def test_same_bits_every_time_on_any_stream_and_in_graphs(D):
    s = _case("bf16", [2000, 37, 515], [65, 65, 65], 8, 2, 128, 32, 64, seed=8)
    d = _cuda(s)
    first = D.tree_attention(*_args(d), mask=d["mask"])["out"]
    for _ in range(3):
        assert torch.equal(D.tree_attention(*_args(d), mask=d["mask"])["out"], first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = D.tree_attention(*_args(d), mask=d["mask"], stream=side)["out"]
    torch.cuda.synchronize()
    assert torch.equal(got, first)
    T, Hq, dim = s["q"].shape
    outs = [torch.empty_like(first) for _ in range(2)]
    ws = torch.zeros(D.attention_workspace_bytes(T, 3, Hq, 2, dim), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, out in zip(graphs, outs):              # two graphs share the workspace, replayed in order
        with torch.cuda.graph(graph):
            D.tree_attention(*_args(d), mask=d["mask"], out=out, workspace=ws)
    d["lengths"].sub_(20)
    want = D.tree_attention(*_args(d), mask=d["mask"])["out"]
    for _ in range(2):
        for graph, out in zip(graphs, outs):
            graph.replay()
            assert torch.equal(out, want)
    assert D.device_error(ws) == 0


@pytest.mark.parametrize("dtype,B,ctx,n,Hq,Hkv,dim,page,N", [
    ("bf16", 24, 1500, 79, 32, 8, 128, 16, 78),       # blocks of 256 rows and blocks of 60 in turn, many per CTA
    ("f16", 40, 900, 33, 28, 4, 64, 32, 32),          # 231 rows a head; ten stages
    ("bf16", 3, 2500, 700, 16, 2, 96, 64, 0),         # causal blocks of growing length
    ("f16", 450, 60, 1, 16, 2, 128, 16, 0),           # more sequences than threads
    ("bf16", 450, 300, 5, 8, 8, 64, 24, 4),
    ("bf16", 1, 60000, 1, 8, 1, 128, 128, 0),         # one block over every CTA
])
def test_many_blocks_per_cta(D, dtype, B, ctx, n, Hq, Hkv, dim, page, N):
    """Enough work that each CTA walks through several blocks, of one half and of two, and joins at both ends."""
    rng = np.random.default_rng(B)
    lengths = [int(x) for x in rng.integers(ctx // 2, ctx + 1, B)]
    s = _case(dtype, lengths, [n] * B, Hq, Hkv, dim, page, N, seed=B)
    d = _cuda(s)
    got = D.tree_attention(*_args(d), mask=d["mask"], lse=True)
    assert D.device_error(got["workspace"]) == 0
    want, lse, bound, lse_bound = refs.attend(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lengths"],
                                              s["starts"], s["mask"], dim ** -0.5, device="cuda")
    refs.close(got["out"], want, bound, s["q"].dtype)
    refs.close(got["lse"], lse, lse_bound, torch.float32)
    for _ in range(3):
        again = D.tree_attention(*_args(d), mask=d["mask"], workspace=got["workspace"])
        assert torch.equal(again["out"], got["out"])


def test_a_wait_that_runs_out_is_reported(D):
    """A limit of 64 cycles ends every wait on memory: the call returns, says so, and the next one is right."""
    s = _case("bf16", [3000, 700], [40, 1], 8, 2, 128, 64, seed=11)
    d = _cuda(s)
    ws = torch.zeros(D.attention_workspace_bytes(41, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    want = D.tree_attention(*_args(d), workspace=ws)["out"]
    flush = torch.ones(64 << 20, dtype=torch.float32, device="cuda")
    D.set_wait_limit(64)
    try:
        flush.mul_(1.0)
        D.tree_attention(*_args(d), workspace=ws)
        flags = D.device_error(ws)
    finally:
        D.set_wait_limit(0)
    assert flags & 1, flags
    assert torch.equal(D.tree_attention(*_args(d), workspace=ws)["out"], want)
    assert D.device_error(ws) == 0


def test_empty_calls(D):
    s = _case("f16", [5], [0], 2, 1, 64, 8, seed=9)
    d = _cuda(s)
    assert D.tree_attention(*_args(d))["out"].shape == (0, 2, 64)


def _tile_columns(S, dim, shift):
    """[S, dim] of 0 and 1: position p of tile t = p // 128 has a 1 in columns t mod a and a + t mod b (a + b <= dim
    without a common factor, so that the pair names the tile), all moved by `shift`."""
    a, b = {64: (31, 33), 96: (47, 49), 128: (61, 67)}[dim]
    t = torch.arange(S) // 128
    assert S <= 128 * a * b
    x = torch.zeros(S, dim, dtype=torch.float64)
    x[torch.arange(S), t % a] = 1.0
    x[torch.arange(S), a + t % b] = 1.0
    return x.roll(shift, 1)


def _uniform(s, D_of_head, skip=None):
    """(out, lse) of equal weights over what each row sees; without tile `skip` = (sequence, tile): a planted mistake."""
    T, Hq, dim = s["q"].shape
    Hkv = s["k_cache"].shape[2]
    N = s["mask"].shape[1] if s["mask"] is not None else 0
    out = torch.full((T, Hq, dim), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    tiles = torch.ones(T, Hq, 1, dtype=torch.float64)
    for b, len_ in enumerate(s["lengths"]):
        at, n = int(s["starts"][b]), int(s["starts"][b + 1] - s["starts"][b])
        S, lead = int(len_) + n, max(n - N, 0)
        if n == 0:
            continue
        see = torch.from_numpy(np.stack([refs.visible(int(len_), n, N, i, s["mask"][b, i - lead] if i >= lead else None)
                                         for i in range(n)])).double()
        if skip is not None and skip[0] == b:
            see[:, 128 * skip[1]:128 * skip[1] + 128] = 0.0
        count = see.sum(-1, keepdim=True)
        for h in range(Hkv):
            rows = (see @ _tile_columns(S, dim, D_of_head * h)) / count
            for g in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                out[at:at + n, g], lse[at:at + n, g] = rows, torch.log(count)[:, 0]
        tiles[at:at + n] = (S + 127) // 128
    return out, lse, tiles


@pytest.mark.parametrize("dtype,lengths,counts,Hq,Hkv,dim,page,N", [
    ("bf16", [60000], [1], 8, 1, 128, 128, 0),           # one block over every CTA
    ("f16", [130000], [1], 4, 1, 64, 64, 0),
    ("bf16", [30000, 77, 12001, 0, 9000], [33, 5, 33, 1, 33], 8, 2, 128, 16, 32),
    ("bf16", [5000], [700], 16, 2, 96, 64, 0),           # causal blocks of growing length
    ("f16", [2900 - 71 * i for i in range(36)], [79] * 36, 8, 2, 128, 16, 78),       # blocks of 256 rows and of 60
])
@pytest.mark.parametrize("scale", [0.0, None])
def test_every_tile_counts_once(D, dtype, lengths, counts, Hq, Hkv, dim, page, N, scale):
    """Equal weights (scale 0, or keys of zeros) over values that name their tile: a tile that is lost or taken twice
    where a span ends, parts are joined or the order turns around changes its columns by a thirtieth or more.

    A weight is 2^x with |x| below 2^-140: 1 within 2^-22, exactly 1 once rounded to 16 bits, so the products' sums are
    whole numbers, exact in fp32.  The sum of weights: 32 additions in a lane's chain, one a tile, one a part, each off
    by at most u; a part's factor 2^-22 and a product, in sum and output alike; 1 / l, its product and a spare u."""
    shift = 7
    s = _case(dtype, lengths, counts, Hq, Hkv, dim, page, N, seed=len(lengths) + dim)
    for b, len_ in enumerate(lengths):
        p = torch.arange(len_ + counts[b])
        where = (torch.from_numpy(s["pages"][b]).long()[p // page], p % page)
        if scale is None:
            s["k_cache"][where] = 0.0
        for h in range(Hkv):
            s["v_cache"][where + (torch.full_like(p, h),)] = _tile_columns(len(p), dim, shift * h).to(DT[dtype])
    d = _cuda(s)
    got = D.tree_attention(*_args(d), mask=d["mask"], scale=scale, lse=True)
    assert D.device_error(got["workspace"]) == 0
    want, lse, tiles = _uniform(s, shift)
    off = 3 * 2.0 ** -22 + (32 + tiles + 2 * 152 + 3) * refs.U
    refs.close(got["out"], want, off * want, DT[dtype])
    near = off[..., 0] + 2.0 ** -22 + 8 * refs.U * lse
    refs.close(got["lse"], lse, near, torch.float32)
    b = int(np.argmax(lengths))
    for tile in (0, lengths[b] // 256, lengths[b] // 128 - 1):            # the check sees a lost tile
        lost, lost_lse, _ = _uniform(s, shift, (b, tile))
        with pytest.raises(AssertionError):
            refs.close(got["out"], lost, off * lost, DT[dtype])
        with pytest.raises(AssertionError):
            refs.close(got["lse"], lost_lse, near, torch.float32)
