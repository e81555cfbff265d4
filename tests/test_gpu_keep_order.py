"""kv_keep's entries that are out of order but would stay where they are (needs a GB300)."""
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


# entry 2 or 300 names the row that it stands at, behind one that names the same row or a later one
@pytest.mark.parametrize("path", [[0, 5, 2], [0, 2, 2], [0, 2, 2, 9], [*range(299), 300, 300], [*range(299), 310, 300]])
@pytest.mark.parametrize("scored", [False, True])
def test_entries_behind_a_larger_one(D, path, scored):
    page, width = 16, len(path)
    k, v, pages = refs.paged(torch.bfloat16, [420], 2, 64, page, seed=width)
    want, err = k.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.rand((1, 2, 430), generator=torch.Generator().manual_seed(width)) + 1
    want_s = s.clone()
    for i, j in enumerate(path):
        if i != j and j > (path[i - 1] if i else -1):
            want[pages[0, (7 + i) // page], (7 + i) % page] = k[pages[0, (7 + j) // page], (7 + j) % page]
            want_s[0, :, 7 + i] = s[0, :, 7 + j]
    want_s[0, :, 7 + width:7 + 400] = 0
    kc, vc, sc = k.cuda(), v.cuda(), s.cuda()
    more = dict(scores=sc, starts=_i32([0, 400])) if scored else {}
    out = D.kv_keep(kc, vc, pages.cuda(), _i32([7]), _i32([path]), _i32([width]), device_err=err, **more)
    assert err.item() == 32
    assert out.tolist() == [7 + width] and torch.equal(kc.cpu(), want)
    assert torch.equal(sc.cpu(), want_s if scored else s)


def test_a_path_that_stays(D):
    """In order, and nothing to move."""
    k, v, pages = refs.paged(torch.bfloat16, [60], 2, 64, 16, seed=1)
    kc, vc, err = k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = D.kv_keep(kc, vc, pages.cuda(), _i32([7]), _i32([[0, 1, 2, 3]]), _i32([4]), device_err=err)
    assert err.item() == 0 and out.tolist() == [11] and torch.equal(kc.cpu(), k) and torch.equal(vc.cpu(), v)
