"""The calls behind a verified tree on a given stream: their values, not their names alone (needs a GB300)."""
import numpy as np
import pytest

from tests import verified_refs as refs
from tests.steps_refs import random_tree

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def D():
    import draft_tree_construction_gb300 as D
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    D.build()
    return D


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def test_given_streams_give_the_same(D):
    """Everything that a call reads is written on the given stream just before it, behind some milliseconds of other
    work: a call that went elsewhere would read what was there before, or leave its outputs unordered."""
    rng, g, tree, lengths = np.random.default_rng(5), torch.Generator().manual_seed(5), 30, [100, 37]
    k, v, pages = refs.paged(torch.bfloat16, [x + tree + 1 for x in lengths], 2, 64, 16, 5)
    trees = [random_tree(tree, 6, rng) for _ in lengths]
    T = 2 * (tree + 1)
    real = dict(logits=(torch.randn(2, tree + 1, 3000, generator=g) * 3).to(torch.bfloat16),
                uniforms=torch.rand(2, tree + 1, generator=g), temperature=torch.tensor([0.8, 0.5]),
                tokens=torch.from_numpy(rng.integers(0, 9, (2, tree)).astype(np.int32)),
                picks=torch.from_numpy(rng.integers(0, 9, (2, tree + 1)).astype(np.int32)),
                parents=torch.from_numpy(np.stack([t[0] for t in trees])), mask=torch.from_numpy(np.stack([t[2] for t in trees])),
                k=k, v=v, pages=pages, lengths=torch.tensor(lengths, dtype=torch.int32),
                starts=torch.tensor([0, tree + 1, T], dtype=torch.int32),
                q=torch.randn(T, 8, 64, generator=g).to(torch.bfloat16), lse=torch.rand(T, 8, generator=g) + 4,
                scores=torch.rand(2, 2, 140, generator=g))
    real = {key: x.cuda() for key, x in real.items()}

    def run(s, **kw):
        drawn = D.sample_logits(s["logits"], s["uniforms"], temperature=s["temperature"], **kw)
        walked = D.tree_accept(s["picks"], s["tokens"], s["parents"], 5, **kw)
        D.attention_weights(s["q"], s["k"], s["pages"], s["lengths"], s["starts"], s["lse"], s["scores"], mask=s["mask"], **kw)
        a = D.kv_keep(s["k"], s["v"], s["pages"], s["lengths"], walked["path"], walked["counts"], **kw)
        b = D.kv_keep(s["k"], s["v"], s["pages"], s["lengths"], walked["path"], walked["counts"], scores=s["scores"],
                      starts=s["starts"], **kw)
        kept = D.kv_evict(s["k"], s["v"], s["pages"], b, s["scores"], 30, first=2, last=8, **kw)
        return [*drawn.values(), *walked.values(), a, b, *kept.values(), s["k"], s["v"], s["scores"]]

    want = run({key: x.clone() for key, x in real.items()})
    assert int(want[3].max()) > 1              # some path goes beyond its root
    blank = {key: torch.zeros_like(x) for key, x in real.items()}
    busy = torch.rand((4096, 4096), device="cuda")
    side = torch.cuda.Stream()
    run({key: x.clone() for key, x in real.items()}, stream=side)             # what is set up once is set up
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-4
        for key, x in blank.items():
            x.copy_(real[key])
    got = run(blank, stream=side)
    assert not side.query()                    # nothing waited for the device
    side.synchronize()
    for x, y in zip(got, want, strict=True):
        assert torch.equal(x, y)
