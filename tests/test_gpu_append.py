"""kv_append against its 64-bit form (needs a GB300)."""
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


def _case(dtype, lengths, counts, Hq, Hkv, dim, page, heads_first=False, extra=0, seed=0):
    """CPU tensors; the rows behind the last sequence are `extra`."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, T = len(lengths), sum(counts) + extra
    qkv = (torch.randn(T, Hq + 2 * Hkv, dim, generator=g) * 2).to(DT[dtype])
    need = [(a + n + page - 1) // page for a, n in zip(lengths, counts)]
    total, width = sum(need) + 2, max(need) + 1
    order = rng.permutation(total)
    pages, at = np.full((B, width), -1, np.int32), 0
    for b, m in enumerate(need):
        pages[b, :m] = order[at:at + m]
        at += m
    shape = (total, Hkv, page, dim) if heads_first else (total, page, Hkv, dim)
    caches = [torch.randn(shape, generator=g).to(DT[dtype]) for _ in range(2)]
    if heads_first:
        caches = [c.transpose(1, 2) for c in caches]
    return dict(qkv=qkv, k_cache=caches[0], v_cache=caches[1], pages=pages,
                lengths=np.array(lengths, np.int32), starts=np.cumsum([0] + list(counts)).astype(np.int32),
                Hq=Hq, Hkv=Hkv, dim=dim, page=page)


def _cuda(s, heads_first=False):
    d = dict(s)
    d["qkv"] = s["qkv"].cuda()
    for c in ("k_cache", "v_cache"):
        t = s[c].transpose(1, 2).contiguous().cuda().transpose(1, 2) if heads_first else s[c].cuda()
        d[c] = t
    for n in ("pages", "lengths", "starts"):
        d[n] = torch.from_numpy(s[n]).cuda()
    Hq, Hkv = s["Hq"], s["Hkv"]
    d["q"], d["k"], d["v"] = d["qkv"][:, :Hq], d["qkv"][:, Hq:Hq + Hkv], d["qkv"][:, Hq + Hkv:]
    return d


def _want(s, freqs, magnitude, interleaved, qw, kw, eps, offsets):
    """q, its bound, k_cache and v_cache in float64 with the k bound on written rows (0 elsewhere)."""
    T = s["qkv"].shape[0]
    Hq, Hkv = s["Hq"], s["Hkv"]
    seq = np.searchsorted(s["starts"][1:], np.arange(T), side="right")
    inside = seq < len(s["lengths"])
    seq = np.minimum(seq, len(s["lengths"]) - 1)
    index = np.arange(T) - s["starts"][seq]
    slot = s["lengths"][seq].astype(np.int64) + index
    pos = s["lengths"][seq].astype(np.int64) + (offsets if offsets is not None else index)
    x = s["qkv"].double()
    q, qb = refs.turn_heads(x[:, :Hq], qw, eps, freqs, magnitude, interleaved, pos)
    k, kb = refs.turn_heads(x[:, Hq:Hq + Hkv], kw, eps, freqs, magnitude, interleaved, pos)
    kc, vc = s["k_cache"].double().clone(), s["v_cache"].double().clone()
    kcb = torch.zeros_like(kc)
    for t in range(T):
        if inside[t]:
            page, row = int(s["pages"][seq[t], slot[t] // s["page"]]), int(slot[t] % s["page"])
            kc[page, row], kcb[page, row], vc[page, row] = k[t], kb[t], x[t, Hq + Hkv:]
    return q, qb, kc, kcb, vc, torch.from_numpy(inside)


CASES = [
    # dtype, lengths, counts, Hq, Hkv, dim, page, rot, interleaved, norm, offsets, heads first, rows behind
    ("bf16", [4097], [1], 32, 8, 128, 64, 128, False, True, False, False, 0),
    ("bf16", [0], [1], 1, 1, 128, 8, 128, False, False, False, False, 0),
    ("f16", [100, 0, 7, 31], [5, 17, 0, 33], 6, 2, 128, 16, 64, True, True, False, False, 5),
    ("bf16", [1000003, 50], [9, 40], 7, 1, 96, 24, 48, False, True, True, True, 3),
    ("f16", [3, 2, 1], [20, 30, 40], 4, 4, 64, 32, 64, True, False, True, False, 0),
    ("bf16", [65, 130], [63, 70], 3, 3, 72, 8, 16, True, True, False, True, 1),       # an odd number of vectors
    ("f16", [9], [300], 2, 1, 8, 8, 0, False, True, False, False, 0),                  # the smallest head, no turn
    ("bf16", [5] * 70, [3] * 70, 8, 2, 128, 16, 128, False, True, False, False, 4),    # more sequences than lanes
    ("f16", [2000000000], [2], 2, 2, 112, 1 << 20, 112, False, False, False, False, 0),  # positions near 2^31
]


@pytest.mark.parametrize("dtype,lengths,counts,Hq,Hkv,dim,page,rot,inter,norm,off,heads_first,extra", CASES)
def test_append_matches_the_definition(D, dtype, lengths, counts, Hq, Hkv, dim, page, rot, inter, norm, off,
                                       heads_first, extra):
    far = lengths[0] > 10 ** 9
    s = _case(dtype, [0] if far else lengths, counts, Hq, Hkv, dim, page if not far else 16, heads_first, extra,
              seed=dim)
    offsets = None
    T = s["qkv"].shape[0]
    if off:
        offsets = np.random.default_rng(1).integers(0, 50, T).astype(np.int32)
    if far:
        # the position alone is far: the cache stays small
        offsets = np.array([lengths[0], 2 ** 31 - 1], np.int32)
    freqs = D.rotary_frequencies(rot, 10000.0, 4.0, 2048) if rot else (None, 1.0)
    g = torch.Generator().manual_seed(3)
    qw = (1 + 0.2 * torch.randn(dim, generator=g)).to(DT[dtype]) if norm else None
    kw = (1 + 0.2 * torch.randn(dim, generator=g)).to(DT[dtype]) if norm else None
    q, qb, kc, kcb, vc, inside = _want(s, freqs[0], freqs[1], inter, qw, kw, 1e-5, offsets)
    d = _cuda(s, heads_first)
    rotary = D.Rotary(freqs[0], magnitude=freqs[1], interleaved=inter) if rot else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T, Hq, dim), 3.0, dtype=DT[dtype], device="cuda")
    got = D.kv_append(d["q"], d["k"], d["v"], d["k_cache"], d["v_cache"], d["pages"], d["lengths"], d["starts"],
                      rotary=rotary, offsets=torch.from_numpy(offsets).cuda() if offsets is not None else None,
                      q_weight=qw.cuda() if norm else None, k_weight=kw.cuda() if norm else None, eps=1e-5, out=out,
                      device_err=err)
    assert int(err) == 0
    refs.close(got[inside.cuda()], q[inside], qb[inside], DT[dtype])
    assert bool((got[~inside.cuda()] == 3.0).all())                       # rows of no sequence stay
    written = (kcb != 0) | (kc != s["k_cache"].double())
    refs.close(torch.where(written, d["k_cache"].cpu().double(), kc).to(DT[dtype]), kc, kcb, DT[dtype])
    assert torch.equal(torch.where(written, s["k_cache"], d["k_cache"].cpu()), s["k_cache"])   # the rest stays
    assert torch.equal(d["v_cache"].cpu().double(), vc)
    # the queries in place, inside the projection's output: the same bits
    d2 = _cuda(s, heads_first)
    D.kv_append(d2["q"], d2["k"], d2["v"], d2["k_cache"], d2["v_cache"], d2["pages"], d2["lengths"], d2["starts"],
                rotary=rotary, offsets=torch.from_numpy(offsets).cuda() if offsets is not None else None,
                q_weight=qw.cuda() if norm else None, k_weight=kw.cuda() if norm else None, eps=1e-5, out=d2["q"])
    assert torch.equal(d2["q"][inside.cuda()], got[inside.cuda()])
    assert torch.equal(d2["k_cache"], d["k_cache"])


def test_keys_and_values_alone(D):
    s = _case("bf16", [30, 2], [4, 9], 0, 2, 64, 16)
    d = _cuda(s)
    assert D.kv_append(None, d["k"], d["v"], d["k_cache"], d["v_cache"], d["pages"], d["lengths"], d["starts"]) is None
    _, _, kc, _, vc, _ = _want(s, None, 1.0, False, None, None, 0.0, None)
    assert torch.equal(d["k_cache"].cpu().double(), kc) and torch.equal(d["v_cache"].cpu().double(), vc)


def test_tokens_that_do_not_fit_write_nothing(D):
    """A page id or a position out of range: an error bit, the query finished, the cache untouched there."""
    s = _case("f16", [10, 10, 10, 10], [8, 8, 8, 8], 4, 2, 64, 8)
    s["pages"][1, 2] = 10 ** 6                        # positions 16, 17 of sequence 1
    s["pages"][2, 1] = -1                             # positions 10 .. 15 of sequence 2
    s["lengths"][3] = -4
    d = _cuda(s)
    before = [d["k_cache"].clone(), d["v_cache"].clone()]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rotary = D.Rotary(D.rotary_frequencies(64)[0])
    got = D.kv_append(d["q"], d["k"], d["v"], d["k_cache"], d["v_cache"], d["pages"], d["lengths"], d["starts"],
                      rotary=rotary, device_err=err)
    assert int(err) == 32
    ok = np.zeros(32, bool)
    ok[0:8] = True
    ok[8:14] = True
    ok[16 + 6:16 + 8] = True
    touched = set()
    for t in np.nonzero(ok)[0]:
        b, slot = t // 8, 10 + t % 8
        touched.add((int(s["pages"][b, slot // 8]), int(slot % 8)))
    changed = (d["v_cache"] != before[1]).any(-1).any(-1).cpu()
    assert {tuple(int(x) for x in i) for i in changed.nonzero()} == touched
    q, qb = refs.turn_heads(s["qkv"][:24, :4].double(), None, 0, rotary.freqs, 1.0, False,
                            np.concatenate([10 + np.arange(8)] * 3))
    refs.close(got[:24], q, qb, torch.float16)


def test_side_stream_and_graph_replay(D):
    s = _case("bf16", [33, 70], [12, 12], 8, 2, 128, 16)
    d, rotary = _cuda(s), D.Rotary(D.rotary_frequencies(128)[0])
    args = lambda x: (x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"], x["pages"], x["lengths"], x["starts"])
    want = D.kv_append(*args(d), rotary=rotary)
    d2 = _cuda(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = D.kv_append(*args(d2), rotary=rotary, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(d2["k_cache"], d["k_cache"])
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.kv_append(*args(d2), rotary=rotary, out=out)
    d2["lengths"].sub_(5)
    d["lengths"].sub_(5)
    graph.replay()
    assert torch.equal(out, D.kv_append(*args(d), rotary=rotary)) and torch.equal(d2["v_cache"], d["v_cache"])


def test_frequencies_are_stretched_between_the_bounds():
    import draft_tree_construction_gb300 as D
    plain, one = D.rotary_frequencies(64)
    f, m = D.rotary_frequencies(64, 10000.0, 8.0, 4096)
    assert one == 1.0 and m == 0.1 * math.log(8.0) + 1
    turns = 4096 * plain / (2 * math.pi)
    assert np.array_equal(f[turns >= 32], plain[turns >= 32]) and np.allclose(f[turns <= 1], plain[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert (f[mid] < plain[mid]).all() and (f[mid] > plain[mid] / 8).all()
    assert np.allclose(D.rotary_frequencies(64, 10000.0, 8.0)[0], plain / 8)


@pytest.mark.parametrize("before,behind", [(3000, 0), (0, 20000), (2500, 9000)])
def test_many_rows_of_no_sequence(D, before, behind):
    """CTAs whose warps have nothing to do next to CTAs that work: the rows outside stay, the sequences' tokens come
    out as they do by themselves, and no copy of the one lands in the shared memory of the other."""
    s = _case("bf16", [37, 5, 90], [60, 1, 83], 32, 8, 128, 16, seed=17)
    d, rotary = _cuda(s), D.Rotary(D.rotary_frequencies(128)[0])
    w = torch.full((128,), 1.25, dtype=torch.bfloat16, device="cuda")
    want = D.kv_append(d["q"], d["k"], d["v"], d["k_cache"], d["v_cache"], d["pages"], d["lengths"], d["starts"],
                       rotary=rotary, q_weight=w, k_weight=w)
    n, T = s["qkv"].shape[0], before + s["qkv"].shape[0] + behind
    for _ in range(3):
        d2 = _cuda(s)
        wide = torch.full((T, 48, 128), math.nan, dtype=torch.bfloat16, device="cuda")
        wide[before:before + n] = d2["qkv"]
        out = torch.full((T, 32, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        D.kv_append(wide[:, :32], wide[:, 32:40], wide[:, 40:], d2["k_cache"], d2["v_cache"], d2["pages"],
                    d2["lengths"], d2["starts"] + before, rotary=rotary, q_weight=w, k_weight=w, out=out)
        assert torch.equal(out[before:before + n], want)
        assert bool((out[:before] == 3.0).all()) and bool((out[before + n:] == 3.0).all())
        assert torch.equal(d2["k_cache"], d["k_cache"]) and torch.equal(d2["v_cache"], d["v_cache"])
