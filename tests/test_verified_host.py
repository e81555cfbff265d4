"""Argument checks of the steps behind a verified tree, without a GPU.

The C entry points refuse before any CUDA call (fake device pointers are never
dereferenced); the binding's checks run on CPU tensors with the device check
replaced, and must raise before the library is called.
"""
import ctypes as C
import math

import numpy as np
import pytest

import draft_tree_construction_gb300 as D
from draft_tree_construction_gb300 import DartError, _steps, _verified
from tests import verified_refs as refs

torch = pytest.importorskip("torch")

OK, INVALID = 0, 1
FAKE = 0x10000000
P = C.c_void_p


@pytest.fixture(scope="module")
def L():
    D.build()
    return D.lib()


def _cache(**over):
    c = _steps._Cache(k=FAKE, v=FAKE, table=FAKE, table_stride=4, table_width=4, pages=9, page=16, heads=2, dim=64,
                      dtype=2)
    for x in "kv":
        for name, st in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(c, f"{x}_{name}_stride", st)
    for key, v in over.items():
        setattr(c, key, v)
    return c


BAD_CACHES = [dict(dtype=0), dict(heads=0), dict(dim=60), dict(dim=136), dict(page=12), dict(pages=-1),
              dict(table_width=1 << 27), dict(table_stride=3), dict(k_page_stride=4), dict(v_row_stride=-8),
              dict(k=FAKE + 8), dict(v=0), dict(table=0)]


def _sample(L, **kw):
    c = dict(logits=FAKE, B=2, R=0, V=100, stride=100, dtype=2, u=FAKE, tokens=FAKE, probs=FAKE)
    c.update(kw)
    return L.dart_logits_sample(P(c["logits"]), c["B"], c["R"], c["V"], c["stride"], c["dtype"], P(c["u"]), None, None,
                                None, None, P(c["tokens"]), P(c["probs"]), None)


def test_sample_argument_checks(L):
    assert _sample(L) == OK and _sample(L, B=0, R=3) == OK
    for kw in (dict(B=-1), dict(R=-1), dict(V=0), dict(V=1 << 24, stride=1 << 24), dict(stride=99),
               dict(stride=(1 << 30) + 1), dict(dtype=3), dict(dtype=-1), dict(B=1 << 16, R=1 << 15),
               dict(R=3, logits=0), dict(R=3, logits=FAKE + 1), dict(R=3, dtype=0, logits=FAKE + 2), dict(R=3, u=0),
               dict(R=3, tokens=0), dict(R=3, probs=0)):
        assert _sample(L, **kw) == INVALID, kw


def _accept(L, **kw):
    c = dict(picks=FAKE, tokens=FAKE, parents=FAKE, B=0, N=10, depth=3, path=FAKE, counts=FAKE, out=FAKE)
    c.update(kw)
    return L.dart_tree_accept(P(c["picks"]), P(c["tokens"]), P(c["parents"]), c["B"], c["N"], c["depth"], P(c["path"]),
                              P(c["counts"]), P(c["out"]), None)


def test_accept_argument_checks(L):
    assert _accept(L) == OK
    for kw in (dict(B=-1), dict(N=-1), dict(N=1025), dict(depth=-1), dict(depth=11), dict(B=1, picks=0),
               dict(B=1, tokens=0), dict(B=1, parents=0), dict(B=1, path=0), dict(B=1, counts=0), dict(B=1, out=0)):
        assert _accept(L, **kw) == INVALID, kw


def _keep(L, cache, **kw):
    c = dict(lengths=FAKE, path=FAKE, stride=5, counts=FAKE, B=0, width=5, out=FAKE)
    c.update(kw)
    return L.dart_kv_keep(C.byref(cache) if cache else None, P(c["lengths"]), P(c["path"]), c["stride"], P(c["counts"]),
                          c["B"], c["width"], P(c["out"]), None, None)


def _evict(L, cache, **kw):
    c = dict(lengths=FAKE, B=0, scores=FAKE, seq=200, head=100, width=64, keep=10, first=2, last=3, index=FAKE, out=FAKE)
    c.update(kw)
    return L.dart_kv_evict(C.byref(cache) if cache else None, P(c["lengths"]), c["B"], P(c["scores"]), c["seq"],
                           c["head"], c["width"], c["keep"], c["first"], c["last"], P(c["index"]), P(c["out"]), None,
                           None)


def _weights(L, cache, **kw):
    c = dict(q=FAKE, ts=256, Hq=4, T=0, B=2, lengths=FAKE, starts=FAKE, mask=0, N=0, scale=0.1, lse=FAKE, scores=FAKE,
             seq=200, head=100, width=64)
    c.update(kw)
    return L.dart_attention_weights(P(c["q"]), c["ts"], 64, c["Hq"], c["T"], c["B"], P(c["lengths"]), P(c["starts"]),
                                    P(c["mask"]), c["N"], c["scale"], C.byref(cache) if cache else None, P(c["lse"]),
                                    P(c["scores"]), c["seq"], c["head"], c["width"], None, None)


@pytest.mark.parametrize("over", BAD_CACHES)
def test_cache_checks(L, over):
    # sequences that share a page table, but no call that launches
    assert _weights(L, _cache()) == OK and _weights(L, _cache(**over)) == INVALID
    assert _keep(L, _cache(**over), B=2) == INVALID and _evict(L, _cache(**over), B=2) == INVALID


def test_keep_argument_checks(L):
    assert _keep(L, _cache()) == OK and _keep(L, None) == INVALID
    for kw in (dict(B=-1), dict(B=65536), dict(width=0), dict(width=-1), dict(B=2, stride=4), dict(stride=-1),
               dict(B=1, lengths=0), dict(B=1, path=0), dict(B=1, counts=0)):
        assert _keep(L, _cache(), **kw) == INVALID, kw
    for over in (dict(pages=0), dict(table_width=0)):
        assert _keep(L, _cache(**over), B=1) == INVALID


def test_values_that_are_the_keys_lie_like_them(L):
    same = _cache()
    same.v, same.v_page_stride, same.v_row_stride, same.v_head_stride = \
        same.k, same.k_page_stride, same.k_row_stride, same.k_head_stride
    assert _keep(L, same) == OK and _evict(L, same) == OK
    for name in ("v_page_stride", "v_row_stride", "v_head_stride"):
        other = _cache()
        other.v = other.k
        for n in ("page", "row", "head"):
            setattr(other, f"v_{n}_stride", getattr(other, f"k_{n}_stride"))
        setattr(other, name, getattr(other, name) + 8)
        assert _keep(L, other) == INVALID and _evict(L, other) == INVALID


def test_evict_argument_checks(L):
    assert _evict(L, _cache()) == OK and _evict(L, None) == INVALID
    for kw in (dict(B=-1), dict(B=65536), dict(width=-1), dict(keep=0), dict(first=-1), dict(last=-1), dict(first=11),
               dict(first=6, last=5), dict(seq=-1), dict(head=-1), dict(head=63), dict(B=2, seq=63),
               dict(B=1, lengths=0), dict(B=1, scores=0), dict(B=1, index=0)):
        assert _evict(L, _cache(), **kw) == INVALID, kw
    for over in (dict(pages=0), dict(table_width=0)):
        assert _evict(L, _cache(**over), B=1) == INVALID


def test_weights_argument_checks(L):
    assert _weights(L, _cache()) == OK and _weights(L, None) == INVALID
    for kw in (dict(Hq=3), dict(Hq=0), dict(Hq=65536), dict(T=-1), dict(T=(1 << 26) + 1), dict(B=-1), dict(N=-1),
               dict(N=1025), dict(scale=math.nan), dict(scale=2.9e38), dict(width=-1), dict(head=63), dict(seq=63),
               dict(T=3, q=0), dict(T=3, q=FAKE + 8), dict(T=3, ts=260), dict(T=3, lengths=0), dict(T=3, starts=0),
               dict(T=3, N=5), dict(T=3, lse=0), dict(T=3, scores=0)):
        assert _weights(L, _cache(), **kw) == INVALID, kw


# --------------------------------------------------------------- the binding

@pytest.fixture
def on_cpu(monkeypatch):
    """CPU tensors pass the device check; a call that reaches the library fails."""
    def reached(*args):
        raise AssertionError("the library was called")
    names = ("dart_logits_sample", "dart_tree_accept", "dart_kv_keep", "dart_attention_weights", "dart_kv_evict")
    stub = type("Stub", (), {name: staticmethod(reached) for name in names})()
    monkeypatch.setattr(_verified, "lib", lambda: stub)
    monkeypatch.setattr(_verified, "_one_device", lambda names, tensors: torch.device("cpu"))
    monkeypatch.setattr(_verified, "_enter", lambda dev, stream: None)
    monkeypatch.setattr(_verified, "_stream", lambda stream, dev: 0)


def _h(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _f(*shape):
    return torch.zeros(shape)


def _raises(call, good, bad):
    with pytest.raises(AssertionError):
        call(**good)
    for kw in bad:
        with pytest.raises(DartError):
            call(**dict(good, **kw))


def test_sample_binding_checks(on_cpu):
    _raises(D.sample_logits, dict(logits=_h(2, 3, 50), uniforms=_f(2, 3), temperature=_f(2), top_k=_i(2), top_p=_f(2),
                                  min_p=_f(2)),
            [dict(logits=_h(6, 50)), dict(logits=_h(2, 3, 50).double()), dict(logits=_h(2, 3, 0)),
             dict(logits=_h(2, 50, 3).transpose(1, 2)), dict(logits=_h(3, 2, 50).transpose(0, 1)),
             dict(uniforms=_f(2, 4)), dict(uniforms=_f(2, 3).double()), dict(uniforms=_f(3, 2).t()),
             dict(temperature=_f(3)), dict(temperature=_i(2)), dict(top_k=_f(2)), dict(top_p=_f(2, 1)),
             dict(min_p=_f(4)[::2])])
    with pytest.raises(AssertionError):        # a padded vocabulary
        D.sample_logits(_h(2, 3, 56)[..., :50], _f(2, 3))


def test_accept_binding_checks(on_cpu):
    _raises(D.tree_accept, dict(picks=_i(2, 9), tokens=_i(2, 8), parents=_i(2, 8), depth=3),
            [dict(picks=_i(2, 8)), dict(picks=_i(2, 9).long()), dict(tokens=_i(8)), dict(tokens=_i(2, 8).long()),
             dict(parents=_i(2, 7)), dict(parents=_i(8, 2).t()), dict(depth=-1), dict(depth=9)])


def _paged():
    return dict(k_cache=_h(5, 16, 2, 64), v_cache=_h(5, 16, 2, 64), pages=_i(2, 3), lengths=_i(2))


BAD_PAGED = [dict(v_cache=_h(5, 16, 2, 32)), dict(k_cache=_h(5, 16, 2, 64).float(), v_cache=_h(5, 16, 2, 64).float()),
             dict(pages=_i(3, 3)), dict(pages=_i(2, 3).long()), dict(lengths=_i(2, 1)), dict(lengths=_i(2).long()),
             dict(k_cache=_h(1, 16, 2, 64).expand(5, 16, 2, 64)), dict(k_cache=_h(5, 12, 2, 64), v_cache=_h(5, 12, 2, 64))]


def test_keep_binding_checks(on_cpu):
    _raises(D.kv_keep, dict(_paged(), path=_i(2, 9)[:, :6], counts=_i(2), device_err=_i(1)),
            BAD_PAGED + [dict(path=_i(2, 0)), dict(path=_i(3, 6)), dict(path=_i(2, 6).long()), dict(path=_i(6, 2).t()),
                         dict(path=_i(1, 6).expand(2, 6)), dict(counts=_i(3)), dict(counts=_f(2)), dict(device_err=_f(1)),
                         dict(device_err=_i(0))])


def test_evict_binding_checks(on_cpu):
    _raises(D.kv_evict, dict(_paged(), scores=_f(2, 2, 48), keep=10, first=4, last=6),
            BAD_PAGED + [dict(scores=_f(2, 3, 48)), dict(scores=_f(2, 48)), dict(scores=_h(2, 2, 48)),
                         dict(scores=_f(2, 48, 2).transpose(1, 2)), dict(scores=_f(2, 1, 48).expand(2, 2, 48)),
                         dict(scores=_f(1, 2, 48).expand(2, 2, 48)), dict(keep=0), dict(first=5), dict(last=-1),
                         dict(device_err=_f(1))])
    with pytest.raises(AssertionError):        # scores kept heads first
        D.kv_evict(**_paged(), scores=_f(2, 2, 48).transpose(0, 1), keep=10)


def test_weights_binding_checks(on_cpu):
    good = dict(_paged(), q=_h(7, 4, 64), starts=_i(3), lse=_f(7, 4), scores=_f(2, 2, 48), mask=_i(2, 40, 2))
    del good["v_cache"]
    bad = [kw for kw in BAD_PAGED if "v_cache" not in kw]
    _raises(D.attention_weights, good,
            bad + [dict(q=_h(7, 3, 64)), dict(q=_h(7, 4, 32)), dict(q=_h(7, 256)), dict(q=_h(7, 4, 64).bfloat16()),
                   dict(q=_h(1, 4, 64).expand(7, 4, 64)), dict(lse=_f(7, 3)), dict(lse=_h(7, 4)), dict(lse=_f(4, 7).t()),
                   dict(starts=_i(2)), dict(starts=_i(3).long()), dict(mask=_i(2, 40, 1)), dict(mask=_i(2, 40)),
                   dict(scores=_f(2, 2, 48).double()), dict(scores=_f(3, 2, 48)), dict(device_err=_f(1))])


def test_host_tensors_are_refused():
    D.build()
    for call in (lambda: D.sample_logits(_h(1, 1, 9), _f(1, 1)), lambda: D.tree_accept(_i(1, 2), _i(1, 1), _i(1, 1), 1),
                 lambda: D.kv_keep(**_paged(), path=_i(2, 3), counts=_i(2)),
                 lambda: D.kv_evict(**_paged(), scores=_f(2, 2, 48), keep=10)):
        with pytest.raises(DartError):
            call()


def test_the_native_module_leaves_what_is_not_on_the_device():
    D.build()
    native = _steps._load_native()
    assert native.sample(1, 2) is None and native.accept() is None and native.keep(None) is None
    assert native.weights(None) is None and native.evict(1, 2, 3) is None
    with pytest.raises(TypeError):
        native.bind_verified(1, 2)


# -------------------------------------------------------------- the references

def test_the_reference_draws_by_hand():
    """Weights 8, 4, 2, 1, 1 in an order of ids that is not theirs."""
    z = np.log([1.0, 8.0, 2.0, 4.0, 1.0])
    draw = lambda u, **kw: refs.sample(z, u, **kw)[0]
    assert [draw(u) for u in (0.0, 0.499, 0.501, 0.74, 0.76, 0.874, 0.876, 0.93, 0.94, 0.999)] == \
        [1, 1, 3, 3, 2, 2, 0, 0, 4, 4]
    assert draw(0.99, k=2) == 3 and draw(0.66, k=2) == 1 and draw(0.67, k=2) == 3
    assert draw(0.99, p=0.5) == 1 and draw(0.99, p=0.51) == 3 and draw(0.99, p=0.76) == 2
    # 12 of the first three's 14 are 0.857
    assert draw(0.99, k=3, p=0.85) == 3 and draw(0.99, k=3, p=0.86) == 2
    assert draw(0.99, m=0.25) == 2 and draw(0.99, m=0.26) == 3 and draw(0.99, m=2.0) == 1
    assert draw(0.99, heat=0.0) == 1 and abs(refs.sample(z, 0.6)[1] - 0.25) < 1e-12
    # half the temperature squares the weights: 64, 16, 4, 1, 1
    assert draw(0.74, heat=0.5) == 1 and draw(0.75, heat=0.5) == 3


def test_the_reference_walks_and_evicts_by_hand():
    assert refs.accept([7, 8, 9, 5], [7, 8, 8], [-1, 0, 0], 3) == ([0, 1, 2], [7, 8, 9])
    assert refs.accept([7, 8, 9, 5], [7, 8, 8], [-1, 0, 0], 1) == ([0, 1], [7, 8])
    assert refs.accept([1, 8, 9, 5], [7, 8, 8], [-1, 0, 0], 3) == ([0], [1])
    s = np.array([0.0, 5.0, 1.0, 5.0, np.nan, 2.0, 9.0])
    assert refs.evict(s, 7, 4, 1, 1) == [0, 1, 3, 6] and refs.evict(s, 7, 3, 0, 0) == [1, 3, 6]
    assert refs.evict(s, 7, 6, 0, 0) == [0, 1, 2, 3, 5, 6] and refs.evict(s, 3, 4, 1, 1) == [0, 1, 2]
