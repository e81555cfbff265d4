"""Argument checks of the steps around a tree, without a GPU.

The C entry points refuse before any CUDA call (fake device pointers are never
dereferenced); the binding's checks run on CPU tensors with the device check
replaced, and must raise before the library is called.
"""
import ctypes as C
import math
from fractions import Fraction

import numpy as np
import pytest

import draft_tree_construction_gb300 as D
from draft_tree_construction_gb300 import DartError, _steps

torch = pytest.importorskip("torch")

OK, INVALID, WORKSPACE = 0, 1, 3
FAKE = 0x10000000
P = C.c_void_p


@pytest.fixture(scope="module")
def L():
    D.build()
    return D.lib()


def _adjust(L, over=None, **kw):
    a = _steps._Adjust(history=FAKE, history_stride=10, history_width=10, repetition=FAKE)
    for key, v in (over or {}).items():
        setattr(a, key, v)
    c = dict(logits=FAKE, B=2, R=0, V=100, stride=100, dtype=2, out=FAKE, out_stride=100)
    c.update(kw)
    return L.dart_logits_adjust(P(c["logits"]), c["B"], c["R"], c["V"], c["stride"], c["dtype"], C.byref(a),
                                P(c["out"]), c["out_stride"], None)


@pytest.mark.parametrize("over,kw,code", [
    ({}, {}, OK), ({}, dict(B=0, R=3), OK),
    ({}, dict(B=-1), INVALID), ({}, dict(B=65536), INVALID), ({}, dict(R=-1), INVALID), ({}, dict(V=0), INVALID),
    ({}, dict(V=1 << 24, stride=1 << 24, out_stride=1 << 24), INVALID), ({}, dict(dtype=3), INVALID),
    ({}, dict(stride=99), INVALID), ({}, dict(out_stride=99), INVALID), ({}, dict(stride=(1 << 30) + 1), INVALID),
    ({}, dict(R=3, logits=0), INVALID), ({}, dict(R=3, out=0), INVALID), ({}, dict(R=3, logits=FAKE + 1), INVALID),
    ({}, dict(R=3, dtype=0, out=FAKE + 2), INVALID), ({}, dict(R=3, out_stride=108), INVALID),   # in place, other rows
    (dict(reserved=1), {}, INVALID), (dict(history_width=-1), {}, INVALID), (dict(history_stride=9), {}, INVALID),
    (dict(bias_count=-1), {}, INVALID), (dict(bias_count=1025), {}, INVALID), (dict(bias_count=4), dict(R=3), INVALID),
    (dict(N=1025), dict(R=1025), INVALID), (dict(N=-1), {}, INVALID), (dict(N=5), dict(R=7), INVALID),
    (dict(N=5), dict(R=4), INVALID), (dict(N=5), dict(R=6), INVALID),                 # a tree without tokens or mask
    (dict(allowed=FAKE, allowed_row_stride=-1), {}, INVALID),
])
def test_adjust_argument_checks(L, over, kw, code):
    assert _adjust(L, over, **kw) == code


def _cache(**over):
    c = _steps._Cache(k=FAKE, v=FAKE, table=FAKE, table_stride=4, table_width=4, pages=9, page=16, heads=2, dim=64,
                      dtype=2)
    for x in "kv":
        for name, st in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(c, f"{x}_{name}_stride", st)
    for key, v in over.items():
        setattr(c, key, v)
    return c


BAD_CACHES = [dict(dtype=0), dict(dtype=3), dict(heads=0), dict(dim=4), dict(dim=60), dict(dim=136), dict(page=12),
              dict(page=0), dict(page=4), dict(pages=-1), dict(table_width=-1), dict(table_width=1 << 27),
              dict(table_stride=3), dict(k_page_stride=4), dict(v_row_stride=-8), dict(k=FAKE + 8), dict(v=0),
              dict(table=0), dict(v_head_stride=1 << 40)]


def _append(L, cache=None, rotary=None, **kw):
    c = dict(q=FAKE, Hq=4, T=0, B=2, lengths=FAKE, starts=FAKE, eps=1e-6, out=FAKE, k=FAKE, v=FAKE, ts=512, qw=0)
    c.update(kw)
    return L.dart_kv_append(P(c["q"]), c["ts"], 64, c["Hq"], P(c["k"]), 512, 64, P(c["v"]), 512, 64, c["T"], c["B"],
                            P(c["lengths"]), P(c["starts"]), None, C.byref(rotary) if rotary else None, P(c["qw"]),
                            None, c["eps"], C.byref(cache) if cache else None, P(c["out"]), 256, 64, None, None)


def _rotary(**over):
    r = _steps._Rotary(FAKE, 1.0, 64, 0, 0)
    for key, v in over.items():
        setattr(r, key, v)
    return r


@pytest.mark.parametrize("over", BAD_CACHES)
def test_cache_checks(L, over):
    assert _append(L, _cache()) == OK and _append(L, _cache(**over)) == INVALID
    assert _attend(L, _cache()) == OK and _attend(L, _cache(**over)) == INVALID


def test_append_argument_checks(L):
    assert _append(L, None) == INVALID
    for kw in (dict(T=-1), dict(B=-1), dict(Hq=-1), dict(eps=-1.0), dict(eps=math.nan), dict(T=3, k=0),
               dict(T=3, v=FAKE + 8), dict(T=3, q=0), dict(T=3, out=0), dict(T=3, ts=511), dict(T=3, lengths=0),
               dict(T=3, starts=0), dict(T=3, qw=FAKE + 2)):
        assert _append(L, _cache(), **kw) == INVALID, kw
    assert _append(L, _cache(), _rotary()) == OK
    for over in (dict(rot=8), dict(rot=72), dict(rot=80), dict(rot=0), dict(turns=0), dict(magnitude=math.inf),
                 dict(interleaved=2), dict(reserved=1)):
        assert _append(L, _cache(), _rotary(**over)) == INVALID, over


def _attend(L, cache=None, **kw):
    c = dict(q=FAKE, Hq=4, T=0, B=2, lengths=FAKE, starts=FAKE, mask=0, N=0, scale=0.1, out=FAKE, ws=FAKE,
             wsb=1 << 40, ts=256)
    c.update(kw)
    return L.dart_tree_attention(P(c["q"]), c["ts"], 64, c["Hq"], c["T"], c["B"], P(c["lengths"]), P(c["starts"]),
                                 P(c["mask"]), c["N"], c["scale"], C.byref(cache) if cache else None, P(c["out"]),
                                 256, 64, None, P(c["ws"]), c["wsb"], None)


def test_attention_argument_checks(L):
    assert _attend(L, None) == INVALID
    for kw in (dict(Hq=3), dict(Hq=0), dict(T=-1), dict(B=-1), dict(N=-1), dict(N=1025), dict(scale=math.nan),
               dict(scale=math.inf), dict(scale=2.9e38), dict(T=3, q=0), dict(T=3, out=FAKE + 8), dict(T=3, ts=260), dict(T=3, lengths=0),
               dict(T=3, starts=0), dict(T=3, N=5)):
        assert _attend(L, _cache(), **kw) == INVALID, kw
    for kw in (dict(ws=0), dict(ws=FAKE + 64), dict(wsb=100)):
        assert _attend(L, _cache(), T=3, **kw) == WORKSPACE, kw
    assert D.attention_workspace_bytes(8, 2, 4, 2, 64) > 0
    for bad in ((-1, 2, 4, 2, 64), (8, -1, 4, 2, 64), (8, 2, 5, 2, 64), (8, 2, 0, 2, 64), (8, 2, 4, 0, 64),
                (8, 2, 4, 2, 60), (8, 2, 4, 2, 136)):
        assert D.attention_workspace_bytes(*bad) == 0, bad


def test_turns_are_exact_fractions(L):
    """turns = frac(f / 2 pi) in units of 2^-64, against rational arithmetic with pi to 100 digits."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706"
                  "7982148086513282306647")
    f = np.array([1.0, 0.5, 1e-4, -1.0, -0.3, 0.0, 2.0 ** -40, 1e-30, 12345.678, 2147483647.5, 5e-324, 6.5])
    turns = np.empty(f.size, np.uint64)
    assert L.dart_rotary_pack_host(f.ctypes.data_as(P), f.size, turns.ctypes.data_as(P)) == OK
    for x, got in zip(f, turns):
        want = Fraction(float(x)) / (2 * pi) * 2 ** 64
        off = (int(got) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Fraction(51, 100), x
    for bad in (math.nan, math.inf, 2.0 ** 31):
        b = np.array([bad])
        assert L.dart_rotary_pack_host(b.ctypes.data_as(P), 1, turns.ctypes.data_as(P)) == INVALID
    assert L.dart_rotary_pack_host(None, 2, turns.ctypes.data_as(P)) == INVALID
    assert L.dart_rotary_pack_host(None, 0, None) == OK


# ------------------------------------------------------------- the binding

@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors pass the device check; reaching the library is a failure."""
    monkeypatch.setattr(_steps, "_one_device", lambda names, tensors: torch.device("cuda", 0))

    def reached(dev, stream):
        raise AssertionError("the checks let this call through")
    monkeypatch.setattr(_steps, "_enter", reached)


def test_host_tensors_are_refused():
    z = torch.zeros(2, 3, 100)
    with pytest.raises(DartError, match="CUDA tensor"):
        D.adjust_logits(z)
    x, c, i = torch.zeros(4, 2, 64).half(), torch.zeros(3, 16, 2, 64).half(), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(DartError, match="CUDA tensor"):
        D.kv_append(x, x, x, c, c, i[None], i, i)
    with pytest.raises(DartError, match="CUDA tensor"):
        D.tree_attention(x, c, c, i[None], i, i)


def test_adjust_binding_checks(on_cpu):
    z = torch.zeros(2, 6, 100)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(s)
    with pytest.raises(AssertionError):                                   # everything in order
        D.adjust_logits(z, history=i32(2, 9), lengths=i32(2), repetition=f32(2), presence=f32(2), frequency=f32(2),
                        bias=(i32(2, 3), f32(2, 3)), allowed=i32(2, 4), tokens=i32(2, 5), mask=i32(2, 5, 1))
    for kw in (dict(history=i32(3, 9)), dict(history=i32(2, 9).long()), dict(history=i32(9, 2).t()),
               dict(history=i32(1, 9).expand(2, 9)), dict(lengths=i32(2)),
               dict(history=i32(2, 9), lengths=i32(3)), dict(repetition=f32(3)), dict(presence=f32(2).double()),
               dict(frequency=f32(2, 1)), dict(bias=(i32(2, 3), None)), dict(bias=(i32(2, 3), f32(2, 4))),
               dict(bias=(i32(3), f32(3))), dict(allowed=i32(2, 3)), dict(allowed=i32(2, 5, 4)),
               dict(allowed=f32(2, 4)), dict(tokens=i32(2, 5)), dict(mask=i32(2, 5, 1)),
               dict(tokens=i32(2, 4), mask=i32(2, 4, 1)), dict(tokens=i32(2, 5), mask=i32(2, 5, 2)),
               dict(out=z.half()), dict(out=torch.zeros(2, 6, 101)), dict(out=torch.zeros(2, 100, 6).transpose(1, 2)),
               dict(out=torch.zeros(1, 6, 100).expand(2, 6, 100))):
        with pytest.raises(DartError):
            D.adjust_logits(z, **kw)
    for bad in (z.double(), z[0], z[..., ::2], torch.zeros(2, 6, 0)):
        with pytest.raises(DartError):
            D.adjust_logits(bad)


def _call_args(T=7, B=2, Hq=4, Hkv=2, dim=64, page=16):
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=h(T, Hq, dim), k=h(T, Hkv, dim), v=h(T, Hkv, dim), k_cache=h(3, page, Hkv, dim),
                v_cache=h(3, page, Hkv, dim), pages=i32(B, 3), lengths=i32(B), starts=i32(B + 1)), h, i32


def test_append_binding_checks(on_cpu):
    a, h, i32 = _call_args()
    with pytest.raises(AssertionError):
        D.kv_append(**a, offsets=i32(7), q_weight=h(64), k_weight=h(64), device_err=i32(1))
    with pytest.raises(AssertionError):
        D.kv_append(**dict(a, q=None))
    bad = [dict(q=h(7, 4, 32)), dict(q=h(6, 4, 64)), dict(q=h(7, 4, 64).bfloat16()), dict(k=h(7, 3, 64)),
           dict(v=h(7, 2, 65)[..., :64]), dict(k=h(7, 2, 68)[..., 4:]), dict(q=h(7, 64, 4).transpose(1, 2)),
           dict(v_cache=h(3, 16, 2, 32)), dict(k_cache=h(3, 16, 2, 64).bfloat16()), dict(pages=i32(3, 3)),
           dict(pages=i32(3, 2).t()), dict(lengths=i32(2).long()), dict(starts=i32(2)), dict(offsets=i32(6)),
           dict(q_weight=h(63)), dict(k_weight=h(64).float()), dict(out=h(7, 4, 63)),
           dict(out=h(1, 4, 64).expand(7, 4, 64)), dict(q=None, out=h(7, 4, 64)), dict(q=None, q_weight=h(64)),
           dict(device_err=h(1)), dict(k_cache=h(3, 12, 2, 64), v_cache=h(3, 12, 2, 64)),
           dict(k_cache=h(1, 16, 2, 64).expand(3, 16, 2, 64))]
    for kw in bad:
        with pytest.raises(DartError):
            D.kv_append(**dict(a, **kw))
    for dim in (60, 136):
        b, _, _ = _call_args(dim=dim)
        with pytest.raises(DartError):
            D.kv_append(**b)


def test_rotary_checks():
    for n in (0, 4, 12, 72):
        with pytest.raises(DartError):
            D.Rotary(np.ones(n), device="cpu")
    for bad in (math.nan, 2.0 ** 32):
        with pytest.raises(DartError):
            D.Rotary(np.full(8, bad), device="cpu")
    with pytest.raises(DartError):
        D.Rotary(np.ones(8), magnitude=math.inf, device="cpu")
    for kw in (dict(rot=7), dict(rot=64, base=0.0), dict(rot=64, factor=0.5),
               dict(rot=64, factor=2.0, original=100, fast=1.0, slow=1.0)):
        with pytest.raises(DartError):
            D.rotary_frequencies(**kw)


def test_attention_binding_checks(on_cpu):
    a, h, i32 = _call_args()
    del a["k"], a["v"]
    with pytest.raises(AssertionError):
        D.tree_attention(**a, mask=i32(2, 40, 2), out=h(7, 4, 64), workspace=torch.zeros(1 << 28, dtype=torch.uint8))
    bad = [dict(q=h(7, 3, 64)), dict(q=h(7, 0, 64)), dict(q=h(7, 4, 64).float()), dict(q=h(4, 64)),
           dict(mask=i32(2, 40, 1)), dict(mask=i32(3, 40, 2)), dict(mask=i32(2, 40)), dict(mask=h(2, 40, 2)),
           dict(out=h(7, 4, 32)), dict(out=a["q"]), dict(out=h(7, 1, 64).expand(7, 4, 64)), dict(pages=i32(2)),
           dict(lengths=i32(2, 1)), dict(starts=i32(4)), dict(workspace=torch.zeros(100, dtype=torch.uint8))]
    for kw in bad:
        with pytest.raises(DartError):
            D.tree_attention(**dict(a, **kw))


def test_the_native_module_leaves_what_is_not_on_the_device():
    D.build()
    native = _steps._load_native()
    assert native.adjust(1, 2) is None and native.append() is None and native.attend(None) is None
    with pytest.raises(TypeError):
        native.bind(1, 2)


@pytest.mark.parametrize("content", [None, b"not a shared object"])
def test_without_the_native_module_the_binding_takes_every_call(monkeypatch, tmp_path, content):
    """A module that is missing or cannot be imported is said once; the calls go on."""
    D.build()
    path = tmp_path / "native.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(_steps, "native_path", lambda: str(path))
    monkeypatch.setattr(_steps, "_native", None)
    with pytest.warns(RuntimeWarning, match="longer"):
        native = _steps._load_native()
    assert _steps._native is native
    assert native.adjust(*range(12)) is None and native.append(*range(16)) is None and native.attend(*range(11)) is None
