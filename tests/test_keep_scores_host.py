"""Argument checks of kv_keep with scores, without a GPU (fake device pointers are never dereferenced)."""
import ctypes as C

import pytest

import draft_tree_construction_gb300 as D
from draft_tree_construction_gb300 import DartError, _steps, _verified

torch = pytest.importorskip("torch")

OK, INVALID = 0, 1
FAKE = 0x10000000
P = C.c_void_p


def _cache(**over):
    c = _steps._Cache(k=FAKE, v=FAKE, table=FAKE, table_stride=4, table_width=4, pages=9, page=16, heads=2, dim=64,
                      dtype=2)
    for x in "kv":
        for name, st in (("page", 2048), ("row", 128), ("head", 64)):
            setattr(c, f"{x}_{name}_stride", st)
    for key, v in over.items():
        setattr(c, key, v)
    return c


def _keep(cache, **kw):
    c = dict(lengths=FAKE, path=FAKE, stride=5, counts=FAKE, B=0, width=5, starts=FAKE, scores=FAKE, seq=200, head=100,
             scores_width=64, out=FAKE)
    c.update(kw)
    return D.lib().dart_kv_keep_scored(C.byref(cache) if cache else None, P(c["lengths"]), P(c["path"]), c["stride"],
                                       P(c["counts"]), c["B"], c["width"], P(c["starts"]), P(c["scores"]), c["seq"],
                                       c["head"], c["scores_width"], P(c["out"]), None, None)


def test_argument_checks():
    D.build()
    assert _keep(_cache()) == OK and _keep(None) == INVALID
    for kw in (dict(B=-1), dict(B=65536), dict(width=0), dict(B=2, stride=4), dict(B=1, lengths=0), dict(B=1, path=0),
               dict(B=1, counts=0), dict(B=1, starts=0), dict(B=1, scores=0), dict(scores_width=-1), dict(seq=-1),
               dict(head=-1), dict(head=63), dict(B=2, seq=63)):
        assert _keep(_cache(), **kw) == INVALID, kw
    for over in (dict(pages=0), dict(table_width=0)):
        assert _keep(_cache(**over), B=1) == INVALID
    for over in (dict(dtype=0), dict(dim=60), dict(page=12), dict(table_width=1 << 27), dict(k=FAKE + 8)):
        assert _keep(_cache(**over), B=1) == INVALID


def _h(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _f(*shape):
    return torch.zeros(shape)


def test_binding_checks(monkeypatch):
    """What is wrong is refused before the library is called, and a call goes to the entry point with the scores."""
    called = []
    stub = type("Stub", (), {"dart_kv_keep": staticmethod(lambda *a: called.append(("plain", len(a))) or 0),
                             "dart_kv_keep_scored": staticmethod(lambda *a: called.append(("scored", len(a))) or 0)})()
    monkeypatch.setattr(_verified, "lib", lambda: stub)
    monkeypatch.setattr(_verified, "_one_device", lambda names, tensors: torch.device("cpu"))
    monkeypatch.setattr(_verified, "_enter", lambda dev, stream: None)
    monkeypatch.setattr(_verified, "_stream", lambda stream, dev: 0)
    good = dict(k_cache=_h(5, 16, 2, 64), v_cache=_h(5, 16, 2, 64), pages=_i(2, 3), lengths=_i(2), path=_i(2, 6),
                counts=_i(2), scores=_f(2, 2, 48), starts=_i(3))
    for kw in (dict(scores=None), dict(starts=None), dict(starts=_i(2)), dict(starts=_i(3).long()),
               dict(starts=_i(6)[::2]), dict(scores=_f(2, 3, 48)), dict(scores=_f(2, 48)), dict(scores=_f(2, 2, 48).double()),
               dict(scores=_f(2, 48, 2).transpose(1, 2)), dict(scores=_f(2, 1, 48).expand(2, 2, 48)),
               dict(scores=_f(1, 2, 48).expand(2, 2, 48))):
        with pytest.raises(DartError):
            D.kv_keep(**dict(good, **kw))
    assert not called
    D.kv_keep(**good)
    D.kv_keep(**dict(good, scores=_f(2, 2, 48).transpose(0, 1)))                 # kept heads first
    D.kv_keep(**dict(good, scores=None, starts=None))
    assert called == [("scored", 15)] * 2 + [("plain", 10)]


def test_host_tensors_are_refused():
    D.build()
    with pytest.raises(DartError):
        D.kv_keep(_h(5, 16, 2, 64), _h(5, 16, 2, 64), _i(2, 3), _i(2), _i(2, 3), _i(2), scores=_f(2, 2, 48), starts=_i(3))
