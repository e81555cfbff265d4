"""Sizes that the C entry points' 32-bit integers cannot hold are refused, without a GPU: meta tensors have sizes and
strides and no memory."""
import pytest

import draft_tree_construction_gb300 as D
from draft_tree_construction_gb300 import DartError, _verified

torch = pytest.importorskip("torch")

BIG = (1 << 32) + 5                            # 5 in the lower 32 bits


def _m(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


def _h(*shape):
    return _m(*shape, dtype=torch.float16)


def _f(*shape):
    return _m(*shape, dtype=torch.float32)


def _paged(pages=(2, 3), B=2):
    return dict(k_cache=_h(5, 16, 2, 64), v_cache=_h(5, 16, 2, 64), pages=_m(*pages), lengths=_m(B))


CALLS = {
    "sample rows": (lambda: D.sample_logits(_h(1, BIG, 2), _f(1, BIG))),
    "sample sequences": (lambda: D.sample_logits(_h(BIG, 1, 2), _f(BIG, 1))),
    "sample tokens": (lambda: D.sample_logits(_h(1, 1, BIG), _f(1, 1))),
    "accept": (lambda: D.tree_accept(_m(BIG, 2), _m(BIG, 1), _m(BIG, 1), 1)),
    "accept nodes": (lambda: D.tree_accept(_m(1, BIG + 1), _m(1, BIG), _m(1, BIG), 1)),
    "keep": (lambda: D.kv_keep(**_paged(), path=_m(2, BIG), counts=_m(2))),
    "keep scores": (lambda: D.kv_keep(**_paged(), path=_m(2, 3), counts=_m(2), scores=_f(2, 2, BIG), starts=_m(3))),
    "keep sequences": (lambda: D.kv_keep(**_paged((BIG, 3), BIG), path=_m(BIG, 3), counts=_m(BIG))),
    "pages": (lambda: D.kv_keep(**_paged((2, BIG)), path=_m(2, 3), counts=_m(2))),
    "weights scores": (lambda: D.attention_weights(_h(7, 4, 64), _h(5, 16, 2, 64), _m(2, 3), _m(2), _m(3), _f(7, 4),
                                                   _f(2, 2, BIG))),
    "weights tokens": (lambda: D.attention_weights(_h(BIG, 4, 64), _h(5, 16, 2, 64), _m(2, 3), _m(2), _m(3), _f(BIG, 4),
                                                   _f(2, 2, 48))),
    "evict scores": (lambda: D.kv_evict(**_paged(), scores=_f(2, 2, BIG), keep=10)),
    "evict keep": (lambda: D.kv_evict(**_paged(), scores=_f(2, 2, 48), keep=BIG)),
    "evict last": (lambda: D.kv_evict(**_paged(), scores=_f(2, 2, 48), keep=BIG, last=BIG - 4)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_refused(monkeypatch, name):
    def reached(*args):
        raise AssertionError("the library was called")
    names = ("dart_logits_sample", "dart_tree_accept", "dart_kv_keep", "dart_kv_keep_scored", "dart_attention_weights",
             "dart_kv_evict")
    stub = type("Stub", (), {n: staticmethod(reached) for n in names})()
    monkeypatch.setattr(_verified, "lib", lambda: stub)
    monkeypatch.setattr(_verified, "_one_device", lambda names, tensors: torch.device("meta"))
    monkeypatch.setattr(_verified, "_enter", lambda dev, stream: None)
    monkeypatch.setattr(_verified, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 4096)
    with pytest.raises(DartError):
        CALLS[name]()


def test_an_ordinary_call_reaches_the_library(monkeypatch):
    """With sizes that fit, the same calls come through: it is the sizes that are refused."""
    called = []
    stub = type("Stub", (), {"dart_kv_evict": staticmethod(lambda *a: called.append(a) or 0)})()
    monkeypatch.setattr(_verified, "lib", lambda: stub)
    monkeypatch.setattr(_verified, "_one_device", lambda names, tensors: torch.device("meta"))
    monkeypatch.setattr(_verified, "_enter", lambda dev, stream: None)
    monkeypatch.setattr(_verified, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda self: 4096)
    D.kv_evict(**_paged(), scores=_f(2, 2, 48), keep=10)
    assert len(called) == 1
