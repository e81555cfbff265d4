"""sample_logits against its 64-bit form (needs a GB300)."""
import math

import numpy as np
import pytest

from tests import verified_refs as refs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _near(V, total):
    """How near to an edge a place may lie, in units of the largest weight, for another token to be drawn.

    A weight is within half a part of 2^-(62 - bits), bits = the length of V, and within 2^-45 of itself, so the sum of
    up to V of them, and a share of a sum, within V / 2 parts and 2^-45 of it.  The place and the edge are both off by
    that, the reference's own sums in 64 bits by less."""
    return 2.0 * (V / 2 * 2.0 ** -(62 - V.bit_length()) + 2.0 ** -45 * total)


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


def _check(D, z, u, heat=None, k=None, p=None, m=None):
    """z [B, R, V] and u [B, R] on the CPU, the settings as lists over B; a share of 2^-8 of the rows at most lies too
    near an edge to say."""
    B, R, V = z.shape
    f = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda")
    zc = z.cuda() if z.is_contiguous() else torch.empty_strided(z.shape, z.stride(), dtype=z.dtype, device="cuda").copy_(z)
    out = D.sample_logits(zc, u.cuda(), temperature=f(heat), top_p=f(p), min_p=f(m),
                          top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda"))
    tokens, probs = out["tokens"].cpu(), out["probs"].cpu()
    assert tokens.dtype == torch.int32 and probs.dtype == torch.float32
    unsaid = 0
    for b in range(B):
        rows = z[b].double().numpy()
        one = lambda x, default: default if x is None else float(np.float32(x[b]))
        for r in range(R):
            t, pr, near, total = refs.sample(rows[r], float(u[b, r]), one(heat, 1.0), int(one(k, 0)), one(p, 1.0), one(m, 0.0))
            if near < _near(V, total):
                unsaid += 1
                continue
            assert int(tokens[b, r]) == t, (b, r, near)
            # a quotient of integers, rounded once.  Without limits the sum has the weights that the draw did not have
            # to list in fp32: an exponent y < 64 is off by 2^-24 y (its factor and the product, half a step each), the
            # weight by 2^-24 64 ln 2 = 2^-18.5 of itself, 2^x by 2^-22, a sum of eight by 2^-22.
            off = 2.0 ** -23 + (2.0 ** -18 if k is None and p is None and m is None else 0.0)
            assert abs(float(probs[b, r]) - pr) <= off * pr + 1e-30, (b, r)
    assert unsaid <= max(1, B * R // 256)
    return tokens


def _logits(B, R, V, dtype, seed, scale=2.0, pad=0, spikes=8):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((B, R, V + pad), generator=g) * scale
    ids = torch.randint(0, V, (B, R, spikes), generator=g)
    z.scatter_add_(2, ids, torch.rand((B, R, spikes), generator=g) * 10)
    z[..., V:] = 1e4
    return z.to(DT[dtype])[..., :V], torch.rand((B, R), generator=g)


SETTINGS = {
    "all": {}, "heat": dict(heat=[0.3, 0.8, 1.7]), "greedy": dict(heat=[0.0, -1.0, math.nan]),
    "top_k": dict(k=[1, 5, 40]), "many_k": dict(k=[0, 900, 100000]), "top_p": dict(p=[0.1, 0.9, 0.999]),
    "no_p": dict(p=[1.0, 0.0, 2.0]), "min_p": dict(m=[0.05, 0.5, 1.0]), "no_m": dict(m=[0.0, 1.5, -1.0]),
    "each": dict(heat=[0.7, 1.0, 1.3], k=[50, 0, 300], p=[0.8, 0.95, 1.0], m=[0.01, 0.0, 0.1]),
    "k_then_p": dict(heat=[0.9, 2.0, 5.0], k=[20, 200, 2000], p=[0.5, 0.9, 0.99]),
}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("name", list(SETTINGS))
def test_settings(D, dtype, name):
    z, u = _logits(3, 11, 5003, dtype, seed=len(name), pad=5)
    _check(D, z, u, **SETTINGS[name])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 31, 64, 257, 1000, 32000, 151936])
def test_sizes(D, dtype, V):
    R = 3 if V > 10000 else 9
    z, u = _logits(2, R, V, dtype, seed=V, spikes=min(8, V))
    _check(D, z, u, heat=[0.8, 1.1], k=[0, 20], p=[0.95, 0.9])
    _check(D, z, u, m=[0.02, 0.0])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8, 13])
def test_rows_at_any_alignment(D, dtype, pad):
    z, u = _logits(2, 6, 777, dtype, seed=pad, pad=pad)
    _check(D, z, u, heat=[1.0, 0.6], p=[0.97, 1.0])


# values that share a bin: all tiny, all large, one step apart in 32 bits, few distinct ones
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["tiny", "large", "huge", "close", "quantised", "constant", "negative", "signed zeros"])
def test_unusual_values(D, dtype, kind):
    g = torch.Generator().manual_seed(5)
    n = torch.randn((2, 8, 3001), generator=g)
    z = {"tiny": n * 1e-4, "large": n * 300, "huge": n * 3e4, "close": 10 + n * 1e-4, "quantised": (n * 2).round(),
         "constant": torch.full_like(n, 3.25), "negative": -5 - n.abs() * 3,
         "signed zeros": torch.where(n > 0, 0.0, -0.0)}[kind].to(DT[dtype])
    u = torch.rand((2, 8), generator=g)
    _check(D, z, u)
    _check(D, z, u, heat=[0.01, 50.0], p=[0.9, 0.5])
    _check(D, z, u, k=[7, 1500], p=[0.9, 1.0], m=[0.0, 0.2])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_with_nothing_and_with_infinities(D, dtype):
    z, u = _logits(1, 8, 501, dtype, seed=2)
    z = z.clone()
    z[0, 0] = -math.inf                       # a grammar's mask that leaves nothing
    z[0, 1] = math.nan
    z[0, 2, ::2] = -math.inf
    z[0, 3, ::3] = math.nan
    z[0, 4, 7] = math.inf
    z[0, 5, [3, 400]] = math.inf
    z[0, 6, :500] = -math.inf                 # one token left
    z[0, 7, 1:] = torch.finfo(DT[dtype]).min  # a mask of the type's lowest value
    for kw in ({}, dict(p=[0.9]), dict(k=[3], m=[0.1]), dict(heat=[0.0]), dict(heat=[1e-30]), dict(heat=[math.inf]),
               dict(heat=[math.inf], m=[1.0]), dict(heat=[math.inf], p=[0.5])):
        tokens = _check(D, z, u, **kw)
        assert tokens[0, 0] == -1 and tokens[0, 1] == -1 and tokens[0, 4] == 7 and tokens[0, 6] == 500


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [3000, 40000])
def test_numbers_next_to_an_edge(D, dtype, V):
    """Random numbers and shares that fall within some 2^-25 of an edge, where the sum of the many small weights counts
    to its last bits."""
    z = torch.full((1, 40, V), -5.0)
    z[..., 5:V:V // 4] = 5.0
    z = z.to(DT[dtype])
    w = np.exp(z[0, 0].double().numpy() - 5.0)
    large = np.sort(w)[::-1].cumsum()[:3] / w.sum()
    steps = np.arange(40) - 20
    for edge in large:
        u = torch.from_numpy((np.float32(edge) * (1 + steps * 2.0 ** -23)).astype(np.float32))[None]
        _check(D, z, u)
        _check(D, z, torch.full((1, 40), 0.999), p=[float(u[0, 7])])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spread", [0.5, 1.0, 2.0, 3.0, 6.0])
def test_flat_and_peaked_rows(D, dtype, spread):
    """From rows where a few tokens matter to rows where most do; few rows (shared by a cluster's CTAs) and many."""
    for B, R, V in ((2, 2, 151936), (1, 6, 33333), (2, 80, 9001)):
        z, u = _logits(B, R, V, dtype, seed=int(spread * 10), scale=spread)
        for kw in ({}, dict(p=[0.95]), dict(p=[0.995], heat=[1.5]), dict(k=[1500]), dict(k=[3000], p=[0.9]),
                   dict(m=[0.001]), dict(m=[0.0001], p=[0.9]), dict(heat=[8.0], k=[50]), dict(m=[0.02], p=[0.99]),
                   dict(m=[0.05], p=[0.999], heat=[1.5]), dict(k=[1000], p=[0.95], m=[0.001])):
            _check(D, z, u, **{key: x * B for key, x in kw.items()})


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 18, 19, 20, 37, 38, 39, 75, 77, 151, 153, 303, 304, 305, 400])
def test_numbers_of_rows(D, dtype, rows):
    """Rows shared by eight CTAs and by fewer, rows with a CTA each, and rows that CTAs take one after another."""
    z, u = _logits(1, rows, 33000, dtype, seed=rows, scale=1.0)
    _check(D, z, u, p=[0.9])


# rows that their largest tokens decide, rows whose sums reach far down, and both next to one another
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["peaked", "flat", "both", "constant", "quantised"])
def test_many_rows(D, dtype, kind):
    B, R, V = 8, 61, 4001
    z, u = _logits(B, R, V, dtype, seed=11, scale={"peaked": 4.0, "quantised": 2.0}.get(kind, 0.7), pad=3)
    if kind == "both":
        z[:, ::3] *= 5.0
    elif kind == "constant":
        z = torch.full_like(z, -1.5)
    elif kind == "quantised":
        z = z.round()
    _check(D, z, u)
    _check(D, z, u, heat=[0.0, 0.3, 0.8, 1.0, 1.3, 3.0, 50.0, math.inf], k=[0, 40, 2500, 0, 0, 1, 900, 0],
           p=[1.0, 0.9, 1.0, 0.999, 0.95, 0.5, 0.9999, 0.3], m=[0.0, 0.0, 0.0, 0.01, 0.0, 0.2, 1e-5, 0.0])
    _check(D, z, u, heat=[1.0, 0.7] * 4, m=[0.001, 0.05, 0.0, 1.0] * 2)
    _check(D, z, u, k=[1, 7, 129, 500, 1024, 1025, 2048, 4001])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [0.7, 4.0])
def test_more_rows_than_are_in_flight(D, dtype, scale):
    z, u = _logits(8, 81, 4001, dtype, seed=16, scale=scale, pad=1)
    _check(D, z, u)
    _check(D, z, u, heat=[0.0, 0.3, 0.8, 1.0, 1.3, 3.0, 50.0, math.inf], k=[0, 40, 2500, 0, 0, 1, 900, 0],
           p=[1.0, 0.9, 1.0, 0.999, 0.95, 0.5, 0.9999, 0.3], m=[0.0, 0.0, 0.0, 0.01, 0.0, 0.2, 1e-5, 0.0])
    z[:, ::9] = -math.inf
    _check(D, z, u, p=[0.98] * 8)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_many_long_rows(D, dtype):
    """Vocabularies beyond 2^16, and more rows than are in flight at once."""
    B, R, V = 2, 153, 70001
    z, u = _logits(B, R, V, dtype, seed=12, scale=0.8)
    _check(D, z, u, heat=[1.0, 2.0], p=[0.9, 0.99])
    _check(D, z, u, heat=[1.0, 1.2], k=[30000, 200], p=[0.98, 1.0])
    _check(D, z, u, m=[0.0, 0.01])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_many_rows_with_nothing_and_with_infinities(D, dtype):
    z, u = _logits(1, 320, 601, dtype, seed=13, scale=0.7)
    z[0, 0::7] = -math.inf
    z[0, 1::7] = math.nan
    z[0, 2::7, ::2] = -math.inf
    z[0, 3::7, 5] = math.inf
    z[0, 4::7, :600] = -math.inf
    z[0, 5::7, 1:] = torch.finfo(DT[dtype]).min
    for kw in ({}, dict(p=[0.9]), dict(k=[3], m=[0.1]), dict(k=[400]), dict(heat=[0.0]), dict(heat=[math.inf], p=[0.5])):
        tokens = _check(D, z, u, **kw)
        assert tokens[0, 0] == -1 and tokens[0, 1] == -1 and tokens[0, 3] == 5 and tokens[0, 4] == 600


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [5, 310])
def test_ends_of_the_temperatures(D, dtype, rows):
    """The least and largest temperatures, over logits of every size; largest ones that several tokens share."""
    g = torch.Generator().manual_seed(15)
    n = torch.randn((1, rows, 700), generator=g)
    n[..., ::50] = n.max()
    u = torch.rand((1, rows), generator=g)
    for scale in (1.0, 1e4, 1e-4) + (() if dtype == "f16" else (3e37, 1e-30)):
        z = (n * scale).to(DT[dtype])
        for heat in (1e-45, 1e-38, 2e-30, 1e-12, 1e12, 1e30, 3e38, math.inf):
            if (scale < 1e-20 and heat < 1e-20) or (scale > 1e20 and 1e30 < heat < math.inf):
                continue                      # a temperature below 1.5e-30 counts as that, above 1e30 fewer bits are right
            _check(D, z, u, heat=[heat])
            _check(D, z, u, heat=[heat], p=[0.7], k=[300])


def test_many_rows_replayed(D):
    """A captured call of rows of both sorts follows its inputs, and draws the same every time."""
    z, u = _logits(2, 200, 9001, "bf16", seed=14, scale=0.7)
    z, u = z.cuda(), u.cuda()
    p = torch.tensor([0.95, 0.5], device="cuda")
    heat = torch.ones(2, device="cuda")
    g = torch.cuda.CUDAGraph()
    D.sample_logits(z, u, temperature=heat, top_p=p)
    with torch.cuda.graph(g):
        out = D.sample_logits(z, u, temperature=heat, top_p=p)
    for turn in range(4):
        u.copy_(u.roll(1, 1))
        z.mul_(1.25)
        heat.mul_(0.9)
        want = D.sample_logits(z, u, temperature=heat, top_p=p)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["tokens"], want["tokens"]) and torch.equal(out["probs"], want["probs"])
        assert int(out["tokens"].min()) >= 0


def test_ends_of_the_uniforms(D):
    z, _ = _logits(1, 6, 4000, "bf16", seed=3)
    u = torch.tensor([[0.0, 1.0 - 2.0 ** -24, 1.0, -1.0, 2.0, math.nan]])
    out = D.sample_logits(z.cuda(), u.cuda(), top_p=torch.tensor([0.9], device="cuda"))
    got = out["tokens"].cpu()[0].tolist()
    rows = z[0].double().numpy()
    clamp = [0.0, 1.0 - 2.0 ** -24, 1.0 - 2.0 ** -24, 0.0, 1.0 - 2.0 ** -24, 0.0]
    assert got == [refs.sample(rows[i], clamp[i], p=float(np.float32(0.9)))[0] for i in range(6)]


def test_draws_follow_the_distribution(D):
    """65536 evenly spaced numbers over one row: each token is drawn as often as its weight says, within one."""
    z, _ = _logits(1, 1, 300, "f32", seed=9, scale=1.0, spikes=1)
    n = 1 << 16
    rows = z.expand(1, n, 300).contiguous().cuda()
    u = ((torch.arange(n) + 0.5) / n)[None].cuda()
    tokens = D.sample_logits(rows, u)["tokens"].cpu()[0].numpy()
    p = torch.softmax(z[0, 0].double(), -1).numpy()
    assert np.all(np.abs(np.bincount(tokens, minlength=300) - p * n) <= 1.0 + 1e-6 * n)


def test_empty_and_refusals(D):
    z, u = _logits(2, 3, 50, "bf16", seed=1)
    z, u = z.cuda(), u.cuda()
    assert D.sample_logits(z[:0], u[:0])["tokens"].shape == (0, 3)
    for bad in (dict(uniforms=u.double()), dict(uniforms=u[:, :2]), dict(logits=z.double()), dict(logits=z[0]),
                dict(top_k=torch.ones(2, device="cuda")), dict(temperature=torch.ones(3, device="cuda")),
                dict(min_p=torch.ones(2))):
        kw = dict(logits=z, uniforms=u)
        kw.update(bad)
        with pytest.raises(D.DartError):
            D.sample_logits(kw.pop("logits"), kw.pop("uniforms"), **kw)


def test_stream_and_graph(D):
    z, u = _logits(4, 5, 9000, "f16", seed=4)
    z, u = z.cuda(), u.cuda()
    p = torch.full((4,), 0.9, device="cuda")
    want = D.sample_logits(z, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = D.sample_logits(z, u, top_p=p, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other["tokens"], want["tokens"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = D.sample_logits(z, u, top_p=p)
    u.copy_(u.flip(0))
    z.copy_(z.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["tokens"], want["tokens"].flip(0))
    assert torch.equal(out["probs"], want["probs"].flip(0))
