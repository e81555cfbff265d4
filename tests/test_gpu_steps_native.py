"""The calls that _steps_native makes against the same calls by the Python binding (needs a GB300).

Both end in the same entry point, so the results are the same bits; what the
native module does not take must come out as the binding's error.
"""
import sys
import types

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


@pytest.fixture
def both(D, monkeypatch):
    """Runs a call natively (it must be taken) and by the binding alone."""
    from draft_tree_construction_gb300 import _steps
    native = _steps._load_native()

    def run(name, call):
        taken = []

        def watch(f):
            def g(*args):
                r = f(*args)
                taken.append(r is not None)
                return r
            return g
        monkeypatch.setattr(_steps, "_native", types.SimpleNamespace(**{name: watch(getattr(native, name))}))
        a = call()
        monkeypatch.setattr(_steps, "_native", types.SimpleNamespace(**{name: lambda *args: None}))
        b = call()
        monkeypatch.setattr(_steps, "_native", native)
        assert taken == [True]
        return a, b
    return run


def _i32(*s, high=50):
    return torch.randint(0, high, s, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,pad", [(torch.float32, 0), (torch.bfloat16, 5), (torch.float16, 8)])
def test_adjust(both, D, dtype, pad):
    B, R, V, N = 3, 6, 1001, 5
    z = torch.randn(B, R, V + pad, device="cuda").to(dtype)[..., :V]
    f = lambda: torch.rand(B, device="cuda") + 0.5
    kw = dict(history=_i32(B, 20)[:, :17], lengths=_i32(B, high=18), repetition=f(), presence=f(), frequency=f(),
              bias=(_i32(B, 9), torch.randn(B, 9, device="cuda")), tokens=_i32(B, N), mask=_i32(B, N, 1, high=31))
    for allowed in (None, _i32(B, 32, high=2 ** 31 - 1), _i32(B, R, 40, high=2 ** 31 - 1)[..., :32]):
        a, b = both("adjust", lambda: D.adjust_logits(z, allowed=allowed, **kw))
        assert a.shape == z.shape and a.dtype == dtype and a.stride() == b.stride()
        assert torch.equal(a.nan_to_num(), b.nan_to_num())
        out = torch.empty(B, R, V + 3, device="cuda", dtype=dtype)[..., :V]
        a, b = both("adjust", lambda: D.adjust_logits(z, allowed=allowed, out=out, **kw))
        assert a is out and b is out
    a, b = both("adjust", lambda: D.adjust_logits(z[:1, :1], allowed=_i32(1, 32)[:1] | -1))
    assert torch.equal(a, z[:1, :1]) and torch.equal(b, a)


def _cached(B=3, T=70, Hq=8, Hkv=2, dim=128, page=16, width=12):
    qkv = torch.randn(T, Hq + 2 * Hkv, dim, device="cuda").bfloat16()
    caches = [torch.randn(B * width, page, Hkv, dim, device="cuda").bfloat16() for _ in range(2)]
    pages = torch.randperm(B * width, device="cuda").int().view(B, width)
    return dict(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + Hkv], v=qkv[:, Hq + Hkv:], k_cache=caches[0], v_cache=caches[1],
                pages=pages, lengths=torch.tensor([3, 0, 77], dtype=torch.int32, device="cuda"),
                starts=torch.tensor([0, 20, 60, 70], dtype=torch.int32, device="cuda"))


def test_append(both, D):
    a = _cached()
    rotary, err = D.Rotary(*D.rotary_frequencies(64), interleaved=True), torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.rand(128, device="cuda").bfloat16()
    for kw in (dict(), dict(rotary=rotary, offsets=_i32(70), q_weight=w, k_weight=w, device_err=err),
               dict(rotary=rotary, out=torch.empty(70, 8, 136, dtype=torch.bfloat16, device="cuda")[..., :128])):
        caches = []

        def call():
            caches.append((a["k_cache"].clone(), a["v_cache"].clone()))
            return D.kv_append(**dict(a, k_cache=caches[-1][0], v_cache=caches[-1][1]), **kw).clone()
        x, y = both("append", call)
        assert torch.equal(x, y)
        for c, d, before in zip(*caches, (a["k_cache"], a["v_cache"])):
            assert torch.equal(c, d) and not torch.equal(c, before)
    assert int(err) == 0


def test_attend(both, D):
    a = _cached()
    del a["k"], a["v"]
    a["q"] = a["q"].contiguous()
    ws = torch.zeros(D.attention_workspace_bytes(70, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    for kw in (dict(), dict(mask=_i32(3, 9, 1, high=2 ** 9), lse=True), dict(scale=0.3, workspace=ws),
               dict(out=torch.empty(70, 8, 136, dtype=torch.bfloat16, device="cuda")[..., :128], workspace=ws)):
        results = []

        def call():
            r = D.tree_attention(**a, **kw)
            results.append(r["out"].clone())
            return r
        x, y = both("attend", call)
        assert torch.equal(*results)
        assert (x["lse"] is None) == (y["lse"] is None) == ("lse" not in kw)
        if x["lse"] is not None:
            assert torch.equal(x["lse"], y["lse"])
        if "out" in kw:
            assert x["out"] is kw["out"]
        if "workspace" in kw:
            assert x["workspace"] is ws
        assert D.device_error(x["workspace"]) == 0


def test_the_current_stream_and_graphs(D):
    z, f = torch.randn(2, 3, 5000, device="cuda"), torch.full((2,), 2.0, device="cuda")
    hist = _i32(2, 30)
    want = D.adjust_logits(z, history=hist, repetition=f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = D.adjust_logits(z, history=hist, repetition=f)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = D.adjust_logits(z, history=hist, repetition=f)
    z.add_(1.0)
    graph.replay()
    assert torch.equal(got, D.adjust_logits(z, history=hist, repetition=f))


def test_references_are_kept_in_balance(D):
    a = _cached()
    q = a["q"].contiguous()
    ws = torch.zeros(D.attention_workspace_bytes(70, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    args = (q, a["k_cache"], a["v_cache"], a["pages"], a["lengths"], a["starts"])
    z = torch.randn(1, 1, 64, device="cuda")
    watched = (*args, ws, out, z, None)
    before = [sys.getrefcount(x) for x in watched[:-1]]
    for _ in range(50):
        D.tree_attention(*args, out=out, workspace=ws)
        D.adjust_logits(z, out=z)
        D.kv_append(q, a["k"], a["v"], *args[1:], out=out)
    assert [sys.getrefcount(x) for x in watched[:-1]] == before


def test_what_is_wrong_raises_as_ever(D):
    from draft_tree_construction_gb300 import DartError
    z, i32, f32 = torch.randn(2, 6, 100, device="cuda"), _i32, lambda *s: torch.zeros(s, device="cuda")
    for kw in (dict(history=i32(3, 9)), dict(history=i32(2, 9).long()), dict(history=i32(9, 2).t()),
               dict(lengths=i32(2)), dict(history=i32(2, 9), lengths=i32(3)), dict(repetition=f32(3)),
               dict(repetition=f32(2).cpu()), dict(presence=f32(2).double()), dict(bias=(i32(2, 3), None)),
               dict(bias=(i32(2, 3), f32(2, 4))), dict(bias=(i32(2, 2000), f32(2, 2000))), dict(allowed=i32(2, 3)),
               dict(allowed=f32(2, 4)), dict(tokens=i32(2, 5)), dict(tokens=i32(2, 4), mask=i32(2, 4, 1)),
               dict(out=z.half()), dict(out=f32(2, 6, 101)), dict(out=f32(1, 6, 100).expand(2, 6, 100))):
        with pytest.raises(DartError):
            D.adjust_logits(z, **kw)
    a = _cached()
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(q=h(70, 8, 64)), dict(k=h(70, 3, 128)), dict(v=h(70, 2, 132)[..., :128][..., 4:]),
               dict(k_cache=a["k_cache"].half()), dict(pages=i32(2, 3)), dict(lengths=i32(3).long()),
               dict(starts=i32(3)), dict(offsets=i32(6)), dict(q_weight=h(64)), dict(out=h(1, 8, 128).expand(70, 8, 128)),
               dict(q=None, out=h(70, 8, 128)), dict(device_err=h(1)), dict(eps=-1.0),
               dict(k_cache=h(1, 16, 2, 128).expand(36, 16, 2, 128))):
        with pytest.raises(DartError):
            D.kv_append(**dict(a, **kw))
    del a["k"], a["v"]
    a["q"] = a["q"].contiguous()
    for kw in (dict(q=h(70, 3, 128)), dict(q=a["q"].float()), dict(mask=i32(3, 40, 1)), dict(mask=i32(2, 40, 2)),
               dict(out=a["q"]), dict(out=h(70, 8, 64)), dict(scale=float("nan")), dict(lengths=i32(3).cpu()),
               dict(workspace=torch.zeros(100, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(DartError):
            D.tree_attention(**dict(a, **kw))


def test_two_threads_on_two_streams(D):
    """Calls that overlap, each thread with its own stream, caches and workspace: the bits of calls by themselves."""
    import threading
    cases = [_cached(), _cached()]
    rotary = D.Rotary(*D.rotary_frequencies(128))
    hist, f = _i32(2, 3000), torch.full((2,), 1.5, device="cuda")
    z = torch.randn(2, 4, 60000, device="cuda")
    tables = [torch.zeros(D.attention_workspace_bytes(70, 3, 8, 2, 128), dtype=torch.uint8, device="cuda")
              for _ in range(2)]

    def step(a, ws):
        q = D.kv_append(**a, rotary=rotary)
        att = D.tree_attention(q, a["k_cache"], a["v_cache"], a["pages"], a["lengths"], a["starts"], workspace=ws)
        return att["out"], D.adjust_logits(z, history=hist, repetition=f)
    want = [step(a, ws) for a, ws in zip(cases, tables)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i] = step(cases[i], tables[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:                        # into the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b, ws in zip(got, want, tables):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and D.device_error(ws) == 0


@pytest.mark.parametrize("code", [1, 3, 4])
def test_a_call_that_fails_is_made_once(D, monkeypatch, code):
    """What an entry point answers is the call's answer: a call that it refuses, or whose launch it reports as failed
    (part of it may have been launched), is not made again by the binding.  In place, a second one would scale, norm
    and turn twice."""
    import ctypes as C

    from draft_tree_construction_gb300 import DartError, _steps
    L, calls, kept = D.lib(), [], []

    def answering(name):
        f = C.CFUNCTYPE(C.c_int, *getattr(L, name).argtypes)(lambda *args: calls.append(name) or code)
        kept.append(f)
        return f
    names = ("dart_logits_adjust", "dart_kv_append", "dart_tree_attention")
    stubs = types.SimpleNamespace(dart_attention_workspace_bytes=L.dart_attention_workspace_bytes,
                                  **{name: answering(name) for name in names})
    a = _cached()
    q = a["q"].contiguous()
    z = torch.randn(2, 3, 500, device="cuda")
    before = [t.clone() for t in (z, q, a["k_cache"], a["v_cache"])]
    monkeypatch.setattr(_steps, "lib", lambda: stubs)
    _steps._load_native()
    monkeypatch.setattr(_steps, "lib", D.lib)
    try:
        for call in (lambda: D.adjust_logits(z, history=_i32(2, 30), repetition=torch.full((2,), 2.0, device="cuda"),
                                             out=z),
                     lambda: D.kv_append(q, a["k"], a["v"], a["k_cache"], a["v_cache"], a["pages"], a["lengths"],
                                         a["starts"], rotary=D.Rotary(*D.rotary_frequencies(128)), out=q),
                     lambda: D.tree_attention(q, a["k_cache"], a["v_cache"], a["pages"], a["lengths"], a["starts"])):
            with pytest.raises(DartError, match=f"\\({code}\\)"):
                call()
    finally:
        _steps._load_native()
    assert calls == list(names)
    for t, was in zip((z, q, a["k_cache"], a["v_cache"]), before):
        assert torch.equal(t, was)
    D.tree_attention(q, a["k_cache"], a["v_cache"], a["pages"], a["lengths"], a["starts"])       # the library again


def _leave_an_error_behind(D):
    """device_error on a capturing stream: refused by the runtime, which remembers the refusal."""
    import ctypes as C

    from draft_tree_construction_gb300 import DartError
    with open("/proc/self/maps") as maps:
        path = next(line.split()[-1] for line in maps if "libcudart.so" in line)
    rt, graph = C.CDLL(path), C.c_void_p()
    side, ws = torch.cuda.Stream(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert rt.cudaStreamBeginCapture(C.c_void_p(side.cuda_stream), C.c_int(2)) == 0           # relaxed
    try:
        with pytest.raises(DartError):
            D.device_error(ws, stream=side)
    finally:
        assert rt.cudaStreamEndCapture(C.c_void_p(side.cuda_stream), C.byref(graph)) != 0     # the capture is void
        rt.cudaGetLastError()                    # of the runtime that PyTorch uses; the library has one of its own
    assert not graph.value


def test_an_older_error_is_not_taken_for_a_failed_launch(D):
    """What another call left behind does not make a call raise that has launched, in place least of all."""
    z, hist = torch.randn(2, 3, 5000, device="cuda"), _i32(2, 30)
    rep = torch.full((2,), 2.0, device="cuda")
    a = _cached()
    a["q"], rotary = a["q"].contiguous(), D.Rotary(*D.rotary_frequencies(128))

    def steps(z, a):
        yield D.adjust_logits(z, history=hist, repetition=rep, out=z)
        yield D.kv_append(**a, rotary=rotary, out=a["q"])
        yield D.tree_attention(*(a[k] for k in ("q", "k_cache", "v_cache", "pages", "lengths", "starts")))["out"]
    copies = lambda: (z.clone(), {k: t.clone() for k, t in a.items()})
    want = list(steps(*copies()))
    z2, a2 = copies()
    made = steps(z2, a2)
    for w in want:
        _leave_an_error_behind(D)
        assert torch.equal(next(made), w)


def test_a_refused_call_leaves_no_error_behind(D):
    """The library's other calls, which launch after device_error was refused, launch and say so."""
    parents = torch.tensor([[-1, 0, 0, 1]], dtype=torch.int32, device="cuda")
    want = D.mask_pack(parents)
    z = torch.randn(4, 3000, device="cuda")
    ids = D.row_topk(z, 1.0, 4)[0]
    _leave_an_error_behind(D)
    assert torch.equal(D.mask_pack(parents), want)
    _leave_an_error_behind(D)
    assert torch.equal(D.row_topk(z, 1.0, 4)[0], ids)


def test_without_the_module(D, monkeypatch):
    """The same bits by the binding alone, and one warning."""
    import warnings

    from draft_tree_construction_gb300 import _steps
    a, z, hist = _cached(), torch.randn(2, 3, 5000, device="cuda"), _i32(2, 30)
    rep = torch.full((2,), 1.5, device="cuda")

    def steps():
        caches = [a["k_cache"].clone(), a["v_cache"].clone()]
        q = D.kv_append(**dict(a, k_cache=caches[0], v_cache=caches[1]))
        att = D.tree_attention(q, *caches, a["pages"], a["lengths"], a["starts"])
        return q, *caches, att["out"], D.adjust_logits(z, history=hist, repetition=rep)
    want = steps()
    monkeypatch.setattr(_steps, "native_path", lambda: None)
    monkeypatch.setattr(_steps, "_native", None)
    with warnings.catch_warnings(record=True) as said:
        warnings.simplefilter("always")
        got = steps()
    assert [w.category for w in said] == [RuntimeWarning] and _steps._native is _steps._LeaveAll
    for x, y in zip(got, want):
        assert torch.equal(x, y)
