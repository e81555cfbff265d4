"""The steps behind a verified tree over many steps: what each position has gathered stays with its token (needs a
GB300)."""
import numpy as np
import pytest

from tests import verified_refs as refs
from tests.steps_refs import U

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


@pytest.mark.parametrize("budget", [0, 9])
def test_scores_stay_with_their_tokens(D, budget):
    """Ten steps with trees, and an eviction after each where there is a budget, against the weights of the same text
    token by token: a position's score is what the accepted tokens behind it gave it, within the sum of the bounds of
    refs.weights and half a step of the score for each addition; behind the length it is 0."""
    B, d, V, Hq, Hkv, dim, page = 3, 3, 500, 4, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *shape: torch.randn(shape, generator=g, device="cuda")
    # a toy target: a token's vectors and the logits that follow it depend on the token alone
    qkv = rnd(V, Hq + 2 * Hkv, dim).to(torch.bfloat16)
    follow = (rnd(V, V) * 2).to(torch.bfloat16)
    W, k = 4, 4
    N = D.num_nodes(d, k, W)
    T = B * (N + 1)
    pages = torch.arange(B * 16, dtype=torch.int32, device="cuda").view(B, 16)
    kc, vc = (torch.zeros((B * 16, page, Hkv, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    scores = torch.zeros((B, Hkv, 16 * page), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(B, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, T + 1, N + 1, dtype=torch.int32, device="cuda")
    last = torch.tensor([3, 100, 499], dtype=torch.int32, device="cuda")
    want, off = np.zeros((B, Hkv, 16 * page)), np.zeros((B, Hkv, 16 * page))
    slots = [[[] for _ in range(Hkv)] for _ in range(B)]         # the token of each position, per head
    jumped = 0
    for step in range(10):
        draft = follow[last.long()][:, None].expand(B, d, V).contiguous() + (rnd(B, d, V) * 0.5).to(torch.bfloat16)
        tree = D.tree_build(draft, 1.0, k, W, 0.0, -10.0)
        chunk = torch.cat([last[:, None], tree["tokens"]], 1)
        x = qkv[chunk.flatten().long()]
        q = D.kv_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, pages, lengths, starts)
        att = D.tree_attention(q, kc, vc, pages, lengths, starts, mask=tree["mask"], lse=True)
        u = torch.rand((B, N + 1), generator=g, device="cuda")
        drawn = D.sample_logits(follow[chunk.long()], u, temperature=torch.full((B,), 0.5, device="cuda"),
                                top_k=_i32([8] * B))
        walk = D.tree_accept(drawn["tokens"], tree["tokens"], tree["parents"], d)
        # the rows that were not accepted give nothing
        path = walk["path"]
        row = torch.where(path >= 0, starts[:-1, None] + path, T).long()
        off_path = torch.ones(T + 1, dtype=torch.bool, device="cuda").index_fill_(0, row.flatten(), False)[:T]
        lse = att["lse"].masked_fill(off_path[:, None], torch.inf)
        D.attention_weights(q, kc, pages, lengths, starts, lse, scores, mask=tree["mask"], device_err=err)
        before = lengths.tolist()
        lengths = D.kv_keep(kc, vc, pages, lengths, path, walk["counts"], scores=scores, starts=starts, device_err=err)
        got = scores.double().cpu().numpy()
        for b in range(B):
            n, L = int(walk["counts"][b]), before[b]
            rows = path[b, :n].tolist()
            jumped += rows != list(range(n))
            for h in range(Hkv):
                slots[b][h] += [int(chunk[b, r]) for r in rows]
            S = L + n
            assert int(lengths[b]) == S
            key = torch.stack([qkv[torch.tensor(slots[b][h], device="cuda"), Hq + h] for h in range(Hkv)], 1).cpu()
            at = [b * (N + 1) + r for r in rows]
            add, bound = refs.weights(q[at].cpu(), key, att["lse"][at].cpu(), dim ** -0.5, L, n)
            want[b, :, :S] += add
            off[b, :, :S] += bound + U * want[b, :, :S]
            assert np.all(np.abs(got[b, :, :S] - want[b, :, :S]) <= off[b, :, :S])
            assert np.all(got[b, :, S:] == 0)
            last[b] = walk["tokens"][b, n - 1]
        if not budget:
            continue
        before = lengths.tolist()
        kept = D.kv_evict(kc, vc, pages, lengths, scores, budget, first=1, last=2, device_err=err)
        lengths = kept["lengths"]
        for b, L in enumerate(before):
            n = min(L, budget)
            for h in range(Hkv):
                old = kept["index"][b, h, :n].tolist()
                assert old == refs.evict(got[b, h], L, budget, 1, 2)
                gone = sorted(set(range(L)) - set(old))
                free = [p for p in old if 1 <= p < L - 2]
                # the text's own weights keep the same, but where they are within the bounds of one another
                assert all(want[b, h, p] + off[b, h, p] >= want[b, h, o] - off[b, h, o] for p in free for o in gone)
                for a in (want, off):
                    a[b, h, :n] = a[b, h, old]
                    a[b, h, n:] = 0
                slots[b][h] = [slots[b][h][p] for p in old]
                text = torch.tensor(slots[b][h], device="cuda")
                where = torch.arange(n, device="cuda")
                assert torch.equal(kc[pages[b].long()].flatten(0, 1)[where, h], qkv[text, Hq + h])
                assert torch.equal(vc[pages[b].long()].flatten(0, 1)[where, h], qkv[text, Hq + Hkv + h])
    assert err.item() == 0
    assert jumped > 0                          # some path left nodes out that lie before its own
