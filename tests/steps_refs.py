"""Plain 64-bit forms of the steps around a tree, on the CPU, with the bounds
that the kernels' arithmetic keeps.

u = 2^-24 is half a step of fp32 (one rounding); a rounding to a 16-bit type is
off by at most torch.finfo(t).eps / 2 relative to the value.
"""
import math

import numpy as np
import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def random_tree(N, width, rng):
    """(parents [N], depths [N], packed ancestor-or-self masks [N, ceil(N/32)] int32) of a random tree,
    numbered depth by depth."""
    depth = [1 + i // width for i in range(N)]
    parents = np.full(N, -1, np.int32)
    bits = np.zeros((N, 32 * ((N + 31) // 32)), np.uint8)
    for i in range(N):
        if depth[i] > 1:
            above = [j for j in range(i) if depth[j] == depth[i] - 1]
            parents[i] = above[rng.integers(len(above))]
            bits[i] = bits[parents[i]]
        bits[i, i] = 1
    return parents, np.array(depth, np.int32), np.packbits(bits, axis=-1, bitorder="little").view(np.int32)


def unpack(words, count):
    w = np.ascontiguousarray(words).view(np.uint32)
    return np.unpackbits(w.view(np.uint8), axis=-1, bitorder="little")[..., :count].astype(bool)


# ------------------------------------------------------------------- adjust

def adjust(z, history=None, lengths=None, rep=None, pres=None, freq=None, bias=None, allowed=None, tokens=None,
           mask=None):
    """(adjusted logits in float64, a bound on the kernel's error before and after its one rounding).

    The kernel does at most 4 + (biases of a token) fp32 operations on values
    that never exceed `size`, each off by at most u of the value it gives."""
    B, R, V = z.shape
    x = z.double().numpy().copy()
    bound = np.zeros_like(x)
    N = tokens.shape[1] if tokens is not None else 0
    penal = any(p is not None for p in (rep, pres, freq))
    for b in range(B):
        base = np.zeros(V)
        if history is not None:
            n = len(history[b]) if lengths is None else max(0, min(int(lengths[b]), len(history[b])))
            for t in history[b][:n]:
                if 0 <= t < V:
                    base[t] += 1
        add, size_add, entries = np.zeros(V), np.zeros(V), np.zeros(V)
        if bias is not None:
            for t, val in zip(bias[0][b], bias[1][b]):
                if 0 <= t < V:
                    add[t] += float(val)
                    size_add[t] += abs(float(val))
                    entries[t] += 1
        for r in range(R):
            cnt = base.copy()
            if N and r >= R - N:
                for j in np.nonzero(unpack(mask[b, r - (R - N)], N))[0]:
                    if 0 <= tokens[b, j] < V:
                        cnt[tokens[b, j]] += 1
            y = x[b, r]
            touched = (cnt > 0) & penal
            ra = float(rep[b]) if rep is not None else 1.0
            p = float(pres[b]) if pres is not None else 0.0
            f = float(freq[b]) if freq is not None else 0.0
            with np.errstate(invalid="ignore"):
                y1 = np.where(touched, np.where(y > 0, y / ra, y * ra), y)
                size = np.abs(y1) + np.where(touched, abs(f) * cnt + abs(p), 0.0) + size_add
                y2 = np.where(touched, y1 - f * cnt - p, y1)
                y2 = np.where(entries > 0, y2 + add, y2)
                bound[b, r] = np.where(touched | (entries > 0), (4 + entries) * U * size, 0.0)
            if allowed is not None:
                words = allowed[b] if allowed.ndim == 2 else allowed[b, r]
                y2 = np.where(unpack(words, V), y2, -math.inf)
            x[b, r] = y2
    return torch.from_numpy(x), torch.from_numpy(bound)


def close(got, want, bound, dtype, extra=0.0):
    """|got - want| <= half a step of the output type + bound; infinities and NaN alike where they are expected.

    Below the smallest normal number (finfo.tiny) the type's steps stop
    shrinking: they are all tiny * eps wide (fp16: 2^-14 * 2^-10 = 2^-24), so
    half a step there is tiny * eps / 2 however small the value."""
    g, w, bound = got.double().cpu(), want.cpu(), bound.cpu()
    finite = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(g[~finite & ~torch.isnan(w)], w[~finite & ~torch.isnan(w)])
    slack = half_step(dtype) * (w.abs() + bound).clamp_min(torch.finfo(dtype).tiny) + bound + extra
    bad = finite & ~((g - w).abs() <= slack)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} off; first at {i}: got {g[i]}, want {w[i]}, "
                             f"allowed {slack[i] if slack.dim() else slack}")


# ------------------------------------------------------------------- append

def turn_heads(x, weight, eps, freqs, magnitude, interleaved, positions):
    """x [T, H, D] float64 -> (normalised and turned heads, error bound before the output rounding).

    The norm: 16 squares and additions per lane, 3 more across lanes (20 u on
    the sum, half of it on its root), one division, one addition, a reciprocal
    root of at most 2 ulp (4 u), two products: below 18 u.  A sine or cosine: 2
    ulp (4 u), its argument rounded once within half a turn (pi u), a product:
    below 9 u.  Two products and a sum: 3 u.  Together below 32 u = 2^-19 of
    |a| + |b|, times the magnitude."""
    y = x.clone()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    out, size = y.clone(), y.abs()
    if freqs is not None:
        half = len(freqs)
        # the angle in doubles: off by less than 2^-53 of it, 2e-7 at position 2^31
        ang = torch.tensor([[math.fmod(float(p) * float(f), 2 * math.pi) for f in freqs] for p in positions],
                           dtype=torch.float64).reshape(len(positions), half)
        cos, sin = (magnitude * torch.cos(ang))[:, None], (magnitude * torch.sin(ang))[:, None]
        lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half),
                                                                                     slice(half, 2 * half))
        a, b = y[..., lo], y[..., hi]
        out[..., lo], out[..., hi] = a * cos - b * sin, b * cos + a * sin
        s = abs(magnitude) * (a.abs() + b.abs())
        size[..., lo] = s
        size[..., hi] = s
    return out, size * 2.0 ** -19


# ------------------------------------------------------------------- attend

def visible(len_, n, N, i, mask_row):
    """Boolean [len_ + n]: what token i of a chunk of n sees."""
    S = len_ + n
    lead = max(n - N, 0)
    see = np.zeros(S, bool)
    if i < lead:
        see[:len_ + i + 1] = True
    else:
        see[:len_ + lead] = True
        see[len_ + lead:] = unpack(mask_row, N)[:n - lead]
    return see


def attend(q, k_cache, v_cache, pages, lengths, starts, mask, scale, device="cpu"):
    """(out, lse, bound on out, bound on lse), float64, for the rows inside sequences; NaN elsewhere.

    A score is a sum of D products accumulated in fp32 with at most 2 u each
    (the tensor unit may cut instead of round): delta = 2 D u scale sum |q||k|,
    and scaling, the maximum's subtraction and the exponential add less than
    2^-20 + 8 u |score - max|.  Each probability is rounded to the 16-bit type (half a step;
    below fp16's normal range 2^-25 absolute against a sum of at least 1), the
    two sums over S positions take 2 u each per term."""
    T, Hq, D = q.shape
    _, page, Hkv, _ = k_cache.shape
    G = Hq // Hkv
    dt = q.dtype
    new = lambda *shape, fill=0.0: torch.full(shape, fill, dtype=torch.float64, device=device)
    out, bound = new(T, Hq, D, fill=math.nan), new(T, Hq, D)
    lse, lse_bound = new(T, Hq, fill=math.nan), new(T, Hq)
    q, k_cache, v_cache = q.to(device), k_cache.to(device), v_cache.to(device)
    N = mask.shape[1] if mask is not None else 0
    for b in range(len(lengths)):
        len_, n, at = int(lengths[b]), int(starts[b + 1] - starts[b]), int(starts[b])
        S = len_ + n
        if n == 0:
            continue
        pos = torch.arange(S)
        rows = torch.as_tensor(pages[b]).long()[pos // page]
        where = (rows.to(device), (pos % page).to(device))
        k = k_cache[where].double().transpose(0, 1)                    # [Hkv, S, D]
        v = v_cache[where].double().transpose(0, 1)
        lead = max(n - N, 0)
        see = np.stack([visible(len_, n, N, i, mask[b, i - lead] if i >= lead else None) for i in range(n)])
        see = torch.from_numpy(see).to(device)                         # [n, S]
        qq = q[at:at + n].double().view(n, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, n * G, D)
        wide = see[None, :, None, :].expand(Hkv, n, G, S).reshape(Hkv, n * G, S)
        s = (qq @ k.transpose(1, 2) * scale).masked_fill(~wide, -math.inf)
        size = (qq.abs() @ k.abs().transpose(1, 2) * abs(scale)).masked_fill(~wide, 0.0).amax(-1, keepdim=True)
        low = s.masked_fill(~wide, math.inf).amin(-1, keepdim=True)
        top = s.amax(-1, keepdim=True)
        some = wide.any(-1, keepdim=True)
        top, low = top.masked_fill(~some, 0.0), low.masked_fill(~some, 0.0)
        w = torch.exp(s - top)
        l = w.sum(-1, keepdim=True)
        p = w / l.clamp_min(1e-300)
        count = see.sum(-1).double()[None, :, None, None].expand(Hkv, n, G, 1).reshape(Hkv, n * G, 1)
        delta = 2 * D * U * size + 2.0 ** -20 + 8 * U * (top - low)
        terms = 2 * U * count
        reach = p @ v.abs()
        eb = (half_step(dt) + 2 * delta + 2 * terms) * reach
        if dt == torch.float16:
            eb = eb + count * 2.0 ** -25 * v.abs().amax()
        back = lambda x: x.view(Hkv, n, G, -1).permute(1, 0, 2, 3).reshape(n, Hq, -1)
        out[at:at + n], bound[at:at + n] = back(p @ v), back(eb)
        sums = (top + torch.log(l)).masked_fill(~some, -math.inf)
        lse[at:at + n] = back(sums)[..., 0]
        lb = delta + terms + 2.0 ** -20 + 4 * U * torch.nan_to_num(sums, neginf=0.0).abs()
        lse_bound[at:at + n] = back(lb)[..., 0]
    return out, lse, bound, lse_bound
