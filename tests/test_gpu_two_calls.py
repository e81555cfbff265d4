"""Calls of other shapes at the same time, from two threads on streams of their own: neither may take from the other
what its launch needs (needs a GB300)."""
import threading

import numpy as np
import pytest

from tests import verified_refs as refs

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


def _together(calls, times):
    """Each call `times` times in a thread and on a stream of its own."""
    errors, ready = [], threading.Barrier(len(calls))

    def work(call):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ready.wait()
                for _ in range(times):
                    call()
            stream.synchronize()
        except BaseException as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_weights_of_other_shapes(D, dim):
    """Blocks of 16, 32 and 112 rows, whose buffers leave other amounts of shared memory."""
    calls, checks = [], []
    for seed, tokens in enumerate((2, 4, 14)):
        lengths = [150, 70]
        g = torch.Generator().manual_seed(seed)
        k, _, pages = refs.paged(torch.bfloat16, [x + tokens for x in lengths], 1, dim, 16, seed)
        kc, pc = k.cuda(), pages.cuda()
        n, starts = _i32(lengths), _i32([0, tokens, 2 * tokens])
        q = torch.randn(2 * tokens, 8, dim, generator=g).to(torch.bfloat16).cuda()
        lse = (torch.rand(2 * tokens, 8, generator=g) + 4).cuda()
        want = D.attention_weights(q, kc, pc, n, starts, lse, torch.zeros((2, 1, 200), device="cuda"))
        got = torch.zeros((2, 1, 200), device="cuda")

        def call(q=q, kc=kc, pc=pc, n=n, starts=starts, lse=lse, got=got):
            got.zero_()
            D.attention_weights(q, kc, pc, n, starts, lse, got)
        calls.append(call)
        checks.append((got, want))
    torch.cuda.synchronize()
    _together(calls, 1000)
    assert all(torch.equal(got, want) for got, want in checks)


@pytest.mark.parametrize("shapes", [[(3, 4, 4), (32, 32, 32)], [(4, 5, 40), (15, 32, 64)]])
def test_trees_of_other_shapes(D, shapes):
    """Frontiers up to 32 and beyond are two kernels; trees of one kernel need other amounts of shared memory.  The C
    entry point by itself: the binding's host work would leave the threads little to meet in."""
    calls, checks = [], []
    for d, k, W in shapes:
        rng = np.random.default_rng(d)
        ids = _i32(np.argsort(rng.random((1, d, 100)), axis=-1)[..., :k])
        logp = torch.from_numpy(np.sort(rng.normal(size=(1, d, k)))[..., ::-1].copy()).cuda()
        want = D.tree_from_topk(ids, logp, W, 0.0, 0.0)
        out = {key: torch.zeros_like(x) for key, x in want.items()}
        outs = [out[key].data_ptr() for key in ("tokens", "parents", "pos", "mask", "scores")]
        build = D.lib().dart_tree_from_topk

        def call(args=(ids.data_ptr(), logp.data_ptr(), 1, d, k, W, 0.0, 0.0, None, None, *outs)):
            stream = torch.cuda.current_stream().cuda_stream
            for _ in range(200):
                rc = build(*args, stream)
                assert rc == 0, rc
        calls.append(call)
        checks.append((out, want))
    torch.cuda.synchronize()
    _together(calls, 100)
    for out, want in checks:
        assert all(torch.equal(out[key], want[key]) for key in want)
