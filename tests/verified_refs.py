"""Plain 64-bit forms of the steps behind a verified tree, on the CPU."""
import math

import numpy as np
import torch

from tests.steps_refs import U, unpack


def sample(z, u, heat=1.0, k=0, p=1.0, m=0.0):
    """(token, probability, distance, sum) of one row: what sample_logits draws, how far a share or u lies from where
    another token would be drawn, and the sum of the weights, both in units of the largest."""
    z = np.asarray(z, np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    order = np.argsort(-z, kind="stable")
    total = int(np.sum(z > -np.inf))
    if total == 0:
        return -1, 0.0, np.inf, 0.0
    order = order[:total]
    if not heat > 0:
        return int(order[0]), 1.0, np.inf, 0.0
    x = z[order]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == x[0], 1.0, 0.0 if np.isinf(x[0]) else np.exp((x - x[0]) / np.float64(heat)))
    n = total if k <= 0 else min(k, total)
    limit = n
    cum = np.cumsum(w)
    near = np.inf
    if p <= 0:
        limit = 1
    elif p < 1:
        limit = min(limit, int(np.searchsorted(cum[:n], p * cum[n - 1])) + 1)
        near = float(np.min(np.abs(cum[:n] - p * cum[n - 1])))
    if m > 0:
        limit = min(limit, int(np.sum(w >= m)))
    limit = max(limit, 1)
    t = u * cum[limit - 1]
    i = min(int(np.searchsorted(cum[:limit], t, side="right")), limit - 1)
    edges = np.abs(cum[:limit - 1] - t)
    if np.all((w == 0.0) | (w == 1.0)):         # sums of whole numbers are exact on both sides
        return int(order[i]), float(w[i] / cum[limit - 1]), np.inf, 0.0
    near = min(near, float(edges.min()) if len(edges) else np.inf)
    return int(order[i]), float(w[i] / cum[limit - 1]), near, float(cum[n - 1])


def accept(picks, tokens, parents, depth):
    path, at = [0], -1
    out = [int(picks[0])]
    while len(path) <= depth:
        for i in range(len(tokens)):
            if parents[i] == at and i > at and tokens[i] >= 0 and tokens[i] == picks[at + 1]:
                at = i
                break
        else:
            break
        path.append(at + 1)
        out.append(int(picks[at + 1]))
    return path, out


def weights(q, key, lse, scale, length, n, mask=None):
    """(sum of the weights [Hkv, S] in float64, a bound on the kernel's error) of one chunk.

    q [n, Hq, D], key [S, Hkv, D], lse [n, Hq].  The product's D terms are added in fp32 by a unit that may cut off
    instead of rounding (2u each), its scaling, the row's sum and their difference are fp32 (3u of their sizes), 2^x is
    off by 2 ulp (4u), and the rows are added one after the other (u each), to the score that was there (u)."""
    S, Hkv, D = key.shape
    Hq = q.shape[1]
    G = Hq // Hkv
    N = 0 if mask is None else mask.shape[0]
    lead = max(n - N, 0)
    seen = np.arange(S)[None, :] <= length + np.arange(n)[:, None]
    if N:
        bits = unpack(mask, N)
        nodes = n - lead
        seen[lead:, :] = False
        seen[lead:, :length + lead] = True
        seen[lead:, length + lead:length + n] = bits[:nodes, :nodes][:, :max(0, S - length - lead)]
    q, key, lse = q.double().numpy(), key.double().numpy(), lse.double().numpy()
    total, bound = np.zeros((Hkv, S)), np.zeros((Hkv, S))
    for h in range(Hkv):
        for g in range(h * G, (h + 1) * G):
            with np.errstate(invalid="ignore", over="ignore"):
                x = q[:, g] @ key[:, h].T * scale
                size = np.abs(q[:, g]) @ np.abs(key[:, h]).T * abs(scale)
                live = seen & np.isfinite(lse[:, g])[:, None]
                y = x - lse[:, g][:, None]
                w = np.where(live, np.exp(np.where(live, y, 0.0)), 0.0)
                off = (2 * D + 3) * U * size + 3 * U * np.abs(np.where(live, lse[:, g][:, None], 0.0)) + 4 * U
                off = np.where(live, off, 0.0)
            total[h] += w.sum(0)
            bound[h] += (w * np.expm1(off)).sum(0)
    return total, bound + (n * G + 4) * U * total


def evict(scores, length, keep, first, last):
    """The kept positions of one head, ascending."""
    if length <= keep:
        return list(range(length))
    s = np.where(np.isnan(scores[:length]), -np.inf, scores[:length])
    free = np.arange(first, length - last)
    # NaN is the least, below -inf
    order = sorted(free, key=lambda i: (bool(np.isnan(scores[i])), -s[i], i))
    return sorted(list(range(first)) + list(range(length - last, length)) + [int(i) for i in order[:keep - first - last]])


def paged(dtype, lengths, heads, dim, page, seed, heads_first=False, spare=2, width_extra=1):
    """(k_cache, v_cache, pages) on the CPU, every sequence's pages in random order."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [max(1, math.ceil(x / page)) for x in lengths]
    total, width = sum(need) + spare, max(need) + width_extra
    order, at = rng.permutation(total), 0
    pages = np.full((len(lengths), width), -1, np.int32)
    for b, m in enumerate(need):
        pages[b, :m] = order[at:at + m]
        at += m
    shape = (total, heads, page, dim) if heads_first else (total, page, heads, dim)
    caches = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
    return caches[0], caches[1], torch.from_numpy(pages)


def rows_of(cache, pages, b, count):
    """[count, heads, dim] of sequence b (cache [pages, page, heads, dim])."""
    page = cache.shape[1]
    p = torch.arange(count)
    return cache[pages[b, p // page].long(), p % page]
