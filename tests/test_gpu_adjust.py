"""adjust_logits against its 64-bit form (needs a GB300)."""
import math

import numpy as np
import pytest

from tests import steps_refs as refs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


def _inputs(dtype, B, R, V, H, K, N, grammar, seed, hot=64):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy(rng.normal(0, 3, (B, R, V)).astype(np.float32)).to(DT[dtype])
    near = lambda shape: np.where(rng.random(shape) < 0.5, rng.integers(0, min(hot, V), shape),
                                  rng.integers(0, V, shape)).astype(np.int32)
    s = dict(z=z, history=near((B, H)), lengths=rng.integers(0, H + 1, B).astype(np.int32),
             rep=rng.uniform(0.8, 1.6, B).astype(np.float32), pres=rng.uniform(-1, 1, B).astype(np.float32),
             freq=rng.uniform(-0.3, 0.5, B).astype(np.float32))
    s["lengths"][0] = H
    if H:
        s["history"][:, ::7] = -1                    # padding among the tokens
        s["history"][0, 1::11] = V                   # and ids behind the vocabulary
    if K:
        ids = near((B, K))
        ids[:, -1] = ids[:, 0]                       # the same token twice
        ids[0, K // 2] = -5
        s["bias"] = (ids, rng.uniform(-6, 6, (B, K)).astype(np.float32))
    if N:
        s["tokens"] = near((B, N))
        trees = [refs.random_tree(N, max(1, N // 6), rng) for _ in range(B)]
        s["mask"] = np.stack([t[2] for t in trees])
        s["tokens"][:, N // 2:] = np.where(rng.random((B, N - N // 2)) < 0.3, s["tokens"][:, :1],
                                           s["tokens"][:, N // 2:])     # the same token again on a path
    if grammar:
        words = (V + 31) // 32
        shape = (B, words) if grammar == "sequence" else (B, R, words)
        w = rng.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32)
        w &= rng.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32)
        w[..., : words // 2] = np.where(rng.random(w[..., : words // 2].shape) < 0.5, 0, 0xFFFFFFFF)
        if grammar == "row":
            w[0, 0] = 0                              # a row that keeps nothing
        else:
            w[-1] = 0
        s["allowed"] = w.view(np.int32)
    return s


def _call(D, s, z, out=None, stream=None, parts=("rep", "pres", "freq")):
    g = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    bias = s.get("bias")
    return D.adjust_logits(z, history=g(s["history"]), lengths=g(s["lengths"]),
                           repetition=g(s["rep"]) if "rep" in parts else None,
                           presence=g(s["pres"]) if "pres" in parts else None,
                           frequency=g(s["freq"]) if "freq" in parts else None,
                           bias=(g(bias[0]), g(bias[1])) if bias else None, allowed=g(s.get("allowed")),
                           tokens=g(s.get("tokens")), mask=g(s.get("mask")), out=out, stream=stream)


def _want(s, parts=("rep", "pres", "freq")):
    return refs.adjust(s["z"], s["history"], s["lengths"], *(s[p] if p in parts else None
                                                             for p in ("rep", "pres", "freq")),
                       s.get("bias"), s.get("allowed"), s.get("tokens"), s.get("mask"))


CASES = [
    # dtype, B, R, V, H, K, N, grammar
    ("bf16", 1, 8, 151936, 300, 0, 0, None),
    ("bf16", 3, 2, 32000, 700, 300, 0, "sequence"),
    ("f16", 5, 3, 32000, 64, 0, 0, "row"),
    ("f32", 2, 4, 20011, 513, 17, 0, "row"),
    ("bf16", 2, 61, 9001, 100, 5, 60, "sequence"),       # odd rows: every alignment; a root and 60 nodes
    ("f16", 2, 33, 8200, 40, 0, 33, None),               # nodes alone
    ("f32", 1, 97, 8192, 0, 3, 96, "row"),
    ("bf16", 1, 1, 1, 4, 1, 0, "row"),                   # one token in the vocabulary
    ("f16", 2, 1, 7, 9, 0, 0, None),
    ("bf16", 2, 3, 8193, 1, 1024, 0, None),              # one token beyond a slice; the most biases
    ("f32", 7, 1, 1023, 5000, 0, 0, "sequence"),
    ("bf16", 1, 1025, 500, 30, 0, 1024, None),           # the widest tree
]


@pytest.mark.parametrize("dtype,B,R,V,H,K,N,grammar", CASES)
def test_adjust_matches_the_definition(D, dtype, B, R, V, H, K, N, grammar):
    s = _inputs(dtype, B, R, V, H, K, N, grammar, seed=V + R)
    want, bound = _want(s)
    z = s["z"].cuda()
    got = _call(D, s, z)
    assert got.shape == z.shape
    refs.close(got, want, bound, DT[dtype])
    assert torch.equal(z.cpu(), s["z"])                                  # the input stays
    again = _call(D, s, z, out=z)                                        # in place, the same bits
    assert again is z and torch.equal(again.view(torch.int8), got.contiguous().view(torch.int8))


@pytest.mark.parametrize("parts", [(), ("rep",), ("pres",), ("freq",)])
def test_each_penalty_alone(D, parts):
    s = _inputs("bf16", 2, 3, 5000, 200, 0, 0, None, seed=5)
    want, bound = _want(s, parts)
    refs.close(_call(D, s, s["z"].cuda(), parts=parts), want, bound, torch.bfloat16)


@pytest.mark.parametrize("dtype,V,pad_in,pad_out", [("bf16", 4001, 7, 0), ("bf16", 4000, 64, 8), ("f16", 999, 1, 2),
                                                    ("f32", 1001, 3, 4)])
def test_padded_rows_and_unlike_alignments(D, dtype, V, pad_in, pad_out):
    s = _inputs(dtype, 2, 5, V, 90, 4, 4, "row", seed=V)
    big = torch.full((2, 5, V + pad_in), math.nan, dtype=DT[dtype], device="cuda")
    big[..., :V] = s["z"].cuda()
    want, bound = _want(s)
    got = _call(D, s, big[..., :V])
    refs.close(got, want, bound, DT[dtype])
    room = torch.full((2, 5, V + pad_out + 1), 7.0, dtype=DT[dtype], device="cuda")
    out = _call(D, s, big[..., :V], out=room[..., 1:V + 1])              # starts one element off
    assert torch.equal(out.contiguous().view(torch.int8), got.contiguous().view(torch.int8))
    edge = torch.cat([room[..., :1], room[..., V + 1:]], -1)
    assert bool((edge == 7.0).all()) and bool(torch.isnan(big[..., V:]).all())


def test_untouched_elements_keep_their_bits(D):
    """NaN (with its payload) and infinities pass where nothing applies; a banned NaN becomes -inf."""
    z = torch.randn(1, 2, 4096).to(torch.bfloat16)
    z[0, :, 5], z[0, :, 6], z[0, :, 7] = math.nan, math.inf, -math.inf
    z.view(torch.int16)[0, :, 8] = 0x7FA5                                # another NaN
    z[0, :, 9] = -0.0
    allowed = np.full((1, 128), 0xFFFFFFFF, np.uint32)
    out = D.adjust_logits(z.cuda(), allowed=torch.from_numpy(allowed.view(np.int32)).cuda())
    assert torch.equal(out.cpu().view(torch.int16), z.view(torch.int16))
    allowed[0, 0] = 0
    out = D.adjust_logits(z.cuda(), allowed=torch.from_numpy(allowed.view(np.int32)).cuda()).cpu()
    assert bool((out[..., :32] == -math.inf).all())
    assert torch.equal(out[..., 32:].view(torch.int16), z[..., 32:].contiguous().view(torch.int16))
    hist = torch.tensor([[5, 6, 7, 9]], dtype=torch.int32, device="cuda")
    out = D.adjust_logits(z.cuda(), history=hist, presence=torch.ones(1, device="cuda")).cpu().float()
    assert math.isnan(out[0, 0, 5]) and out[0, 0, 6] == math.inf and out[0, 0, 7] == -math.inf and out[0, 0, 9] == -1


def test_broadcast_masks_and_strided_histories(D):
    s = _inputs("bf16", 3, 4, 3000, 50, 0, 0, "sequence", seed=2)
    want, bound = _want(s)
    dev = lambda x: torch.from_numpy(x).cuda()
    wide = torch.full((3, 80), 2, dtype=torch.int32, device="cuda")
    wide[:, 10:60] = dev(s["history"])
    rows = dev(s["allowed"])[:, None, :].expand(3, 4, -1)
    got = D.adjust_logits(s["z"].cuda(), history=wide[:, 10:60], lengths=dev(s["lengths"]), repetition=dev(s["rep"]),
                          presence=dev(s["pres"]), frequency=dev(s["freq"]), allowed=rows)
    refs.close(got, want, bound, torch.bfloat16)


def test_empty_batches(D):
    for shape in ((0, 3, 100), (2, 0, 100)):
        z = torch.zeros(shape, dtype=torch.float16, device="cuda")
        assert D.adjust_logits(z).shape == shape


def test_side_stream_and_graph_replay(D):
    """A captured call reads what the buffers hold at each replay."""
    s = _inputs("bf16", 2, 21, 6000, 80, 6, 20, "row", seed=9)
    z = s["z"].cuda()
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    kw = dict(history=dev(s["history"]), lengths=dev(s["lengths"]), repetition=dev(s["rep"]), presence=dev(s["pres"]),
              frequency=dev(s["freq"]), bias=tuple(dev(x) for x in s["bias"]), allowed=dev(s["allowed"]),
              tokens=dev(s["tokens"]), mask=dev(s["mask"]))
    first = D.adjust_logits(z, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = D.adjust_logits(z, stream=side, **kw)
    torch.cuda.synchronize()
    assert torch.equal(got.view(torch.int16), first.view(torch.int16))
    out = torch.empty_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.adjust_logits(z, out=out, **kw)
    z.copy_(torch.randn_like(z))
    kw["lengths"].fill_(3)
    graph.replay()
    assert torch.equal(out.view(torch.int16), D.adjust_logits(z, **kw).view(torch.int16))


@pytest.mark.parametrize("dtype,B,R,V", [("f32", 16, 5, 32000), ("bf16", 7, 3, 1003)])
def test_long_histories(D, dtype, B, R, V):
    """Lengths about the ends of the batches in which a CTA reads them; many rows a CTA and few."""
    s = _inputs(dtype, B, R, V, 15000, 5, 0, None, seed=B)
    s["lengths"][:7] = [0, 1, 2047, 2048, 2049, 6145, 14999]
    got = _call(D, s, s["z"].cuda())
    want, bound = _want(s)
    refs.close(got, want, bound, DT[dtype])


@pytest.mark.parametrize("dtype,V,N,grammar", [("bf16", 9001, 33, None), ("f32", 8192, 5, "row"), ("f16", 1003, 70, None),
                                               ("bf16", 40000, 1000, "sequence")])
def test_what_lies_outside_is_not_counted(D, dtype, V, N, grammar):
    """Tree tokens outside [0, V), mask bits from N up, bias ids outside [0, V): as if they were not there."""
    s = _inputs(dtype, 2, N + 1, V, 50, 12, N, grammar, seed=N)
    far = np.array([-1, -2 ** 31, V, V + 1, 2 ** 31 - 1, V + 65536, -V], np.int64).astype(np.int32)
    rng = np.random.default_rng(N)
    s["tokens"][:, ::3] = rng.choice(far, s["tokens"][:, ::3].shape)
    s["bias"][0][:, 1::2] = rng.choice(far, s["bias"][0][:, 1::2].shape)
    clean = s["mask"].copy()
    if N % 32:
        s["mask"].view(np.uint32)[..., -1] |= np.uint32(0xFFFFFFFF << (N % 32) & 0xFFFFFFFF)
    assert np.array_equal(refs.unpack(s["mask"], N), refs.unpack(clean, N))
    want, bound = _want(s)
    got = _call(D, s, s["z"].cuda())
    refs.close(got, want, bound, DT[dtype])
    # the same bits as a call that names none of it
    inside = dict(s, tokens=s["tokens"].copy(), mask=clean, bias=tuple(x.copy() for x in s["bias"]))
    inside["bias"][0][:, 1::2] = -1
    inside["tokens"][(s["tokens"] < 0) | (s["tokens"] >= V)] = -1
    assert torch.equal(_call(D, inside, s["z"].cuda()).view(torch.int8), got.view(torch.int8))


def test_histories_of_their_own_take_two_calls(D):
    """Repetition over prompt and output, presence and frequency over the output alone: two calls, the second in place."""
    s = _inputs("f32", 2, 4, 5000, 90, 7, 0, "row", seed=31)
    s["history"] = np.abs(s["history"]) % 4000
    prompt, made = s["history"], s["history"][:, 60:]
    g = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    z = D.adjust_logits(s["z"].cuda(), history=g(prompt), repetition=g(s["rep"]))
    got = D.adjust_logits(z, history=g(made), presence=g(s["pres"]), frequency=g(s["freq"]),
                          bias=tuple(g(x) for x in s["bias"]), allowed=g(s["allowed"]), out=z)
    first, bound1 = refs.adjust(s["z"], prompt, None, s["rep"])
    want, bound2 = refs.adjust(first, made, None, None, s["pres"], s["freq"], s["bias"], s["allowed"])
    # the first call's rounding to fp32 enters the second as it stands
    refs.close(got, want, bound2 + bound1 + first.abs() * 2.0 ** -24, torch.float32)


@pytest.mark.parametrize("dtype,B,R,V", [("bf16", 60, 240, 151936), ("f16", 60, 240, 151933), ("f32", 46, 3, 16000003)])
def test_more_elements_than_32_bits_count(D, dtype, B, R, V):
    """Offsets past 2^31 elements (past 2^32 bytes): every sequence as it comes out by itself."""
    assert B * R * V > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(V)
    z = torch.empty(B, R, V, dtype=DT[dtype], device="cuda")
    for b in range(B):
        z[b].normal_(generator=gen)
    draw = lambda high, *s: torch.randint(0, high, s, dtype=torch.int32, device="cuda", generator=gen)
    kw = dict(history=draw(V, B, 40), repetition=torch.rand(B, device="cuda", generator=gen) + 0.6,
              frequency=torch.rand(B, device="cuda", generator=gen), allowed=draw(2 ** 31 - 1, B, (V + 31) // 32))
    ids, vals = draw(V, B, 20), torch.randn(B, 20, device="cuda", generator=gen)
    got = D.adjust_logits(z, bias=(ids, vals), **kw)
    for b in range(B):
        alone = D.adjust_logits(z[b:b + 1].clone(), bias=(ids[b:b + 1], vals[b:b + 1]),
                                **{k: x[b:b + 1].contiguous() for k, x in kw.items()})
        assert torch.equal(got[b].view(torch.int8), alone[0].view(torch.int8)), b
    D.adjust_logits(z, bias=(ids, vals), out=z, **kw)
    for b in range(B):
        assert torch.equal(z[b].view(torch.int8), got[b].view(torch.int8)), b
