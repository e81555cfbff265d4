"""The steps behind a verified tree: sampling, the walk along the drawn tokens, what stays in the cache.

Bindings of dart_logits_sample, dart_tree_accept, dart_kv_keep,
dart_kv_keep_scored, dart_attention_weights and dart_kv_evict
(include/darttree.h); the package exports the public names.
"""
from __future__ import annotations

import ctypes as C

from . import _steps
from . import DartError, _check, _check_error_word, _check_tensor, _mask_dtypes, _row_stride, _torch, lib
from ._steps import (_at, _Cache, _cache, _check_inner, _codes, _enter, _heads, _leave, _one_device, _output,
                     _sequences, _stream)


def declare(L):
    P, i32, i64, f32 = C.c_void_p, C.c_int, C.c_int64, C.c_float
    L.dart_logits_sample.argtypes = [P, i32, i32, i32, i64, i32, P, P, P, P, P, P, P, P]
    L.dart_tree_accept.argtypes = [P, P, P, i32, i32, i32, P, P, P, P]
    L.dart_kv_keep.argtypes = [C.POINTER(_Cache), P, P, i64, P, i32, i32, P, P, P]
    L.dart_kv_keep_scored.argtypes = [C.POINTER(_Cache), P, P, i64, P, i32, i32, P, P, i64, i64, i32, P, P, P]
    L.dart_attention_weights.argtypes = [P, i64, i64, i32, i32, i32, P, P, P, i32, f32, C.POINTER(_Cache), P, P, i64,
                                         i64, i32, P, P]
    L.dart_kv_evict.argtypes = [C.POINTER(_Cache), P, i32, P, i64, i64, i32, i32, i32, i32, P, P, P, P]
    for f in (L.dart_logits_sample, L.dart_tree_accept, L.dart_kv_keep, L.dart_kv_keep_scored, L.dart_attention_weights,
              L.dart_kv_evict):
        f.restype = i32


# The usual calls are made by the native module, as those of the steps around a
# tree are: it returns None for what it leaves to the code here.

_bound = None


def _native():
    global _bound
    module = _steps._native or _steps._load_native()
    if module is not _bound:
        L = lib()
        module.bind_verified(*(C.cast(f, C.c_void_p).value for f in
                               (L.dart_logits_sample, L.dart_tree_accept, L.dart_kv_keep, L.dart_attention_weights,
                                L.dart_kv_evict, L.dart_kv_keep_scored)))
        _bound = module
    return module


_MOST = 2 ** 31 - 1


def _sizes(*counts):
    """Sizes that the entry points take as 32-bit integers, which ctypes would cut to their lower half."""
    if max(counts) > _MOST:
        raise DartError(f"sizes must be at most {_MOST}, got {max(counts)}")


# ----------------------------------------------------------------- sampling

def sample_logits(logits, uniforms, *, temperature=None, top_k=None, top_p=None, min_p=None, stream=None) -> dict:
    """Draws a token from each row of logits (dart_logits_sample).

    logits: CUDA [B, R, V] float32/float16/bfloat16, rows evenly spaced (a view
    of a padded vocabulary serves): a sequence's next token, or the rows of a
    verified tree.  uniforms: float32 [B, R] in [0, 1).  temperature, top_p,
    min_p (float32 [B]) and top_k (int32 [B]) hold for a sequence's rows; each
    may be left out.  A temperature of 0 is greedy; a top_k of 0, a top_p of 1
    and a min_p of 0 are no limits.  Of the tokens in descending order of their
    logits (lower id first), the first that all limits leave are drawn from:
    top_p counts from the top_k renormalised, min_p is relative to the largest.
    Returns tokens (int32 [B, R], -1 where a row has nothing to draw from) and
    probs (float32 [B, R], their probabilities among what was kept)."""
    if stream is None and logits.is_cuda:
        made = _native().sample(logits, uniforms, temperature, top_k, top_p, min_p)
        if made is not None:
            return {"tokens": made[0], "probs": made[1]}
    torch = _torch()
    dev = _one_device(("logits", "uniforms", "temperature", "top_k", "top_p", "min_p"),
                      (logits, uniforms, temperature, top_k, top_p, min_p))
    code = _codes().get(logits.dtype)
    if code is None or logits.dim() != 3:
        raise DartError("logits must be [B, R, V] float32, float16 or bfloat16")
    B, R, V = logits.shape
    if V < 1:
        raise DartError("logits must have at least one token")
    _sizes(B, R, V)
    stride = V if logits.is_contiguous() else _row_stride(logits)
    _check_tensor(uniforms, "uniforms", torch.float32, (B, R))
    for t, name in ((temperature, "temperature"), (top_p, "top_p"), (min_p, "min_p")):
        if t is not None:
            _check_tensor(t, name, torch.float32, (B,))
    if top_k is not None:
        _check_tensor(top_k, "top_k", torch.int32, (B,))
    scope = _enter(dev, stream)
    try:
        tokens = torch.empty((B, R), dtype=torch.int32, device=dev)
        probs = torch.empty((B, R), dtype=torch.float32, device=dev)
        rc = lib().dart_logits_sample(logits.data_ptr(), B, R, V, stride, code, uniforms.data_ptr(), _at(temperature),
                                      _at(top_k), _at(top_p), _at(min_p), tokens.data_ptr(), probs.data_ptr(),
                                      _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_logits_sample")
    return {"tokens": tokens, "probs": probs}


# --------------------------------------------------------------- acceptance

def tree_accept(picks, tokens, parents, depth: int, *, stream=None) -> dict:
    """Walks each tree along the tokens picked at its nodes (dart_tree_accept).

    picks: CUDA int32 [B, N + 1], the root's pick and each node's, as
    sample_logits draws them from a tree's N + 1 rows; tokens, parents: int32
    [B, N], as tree_build returns them; depth: the most nodes accepted (the
    tree's d).  Returns path (int32 [B, depth + 1]: row 0, the root's, then the
    row of each accepted node, -1 behind), counts (int32 [B], entries of the
    path) and tokens (int32 [B, depth + 1]: the accepted tokens and the one that
    follows them, -1 behind)."""
    if stream is None and tokens.is_cuda:
        made = _native().accept(picks, tokens, parents, depth)
        if made is not None:
            return {"path": made[0], "counts": made[1], "tokens": made[2]}
    torch = _torch()
    dev = _one_device(("picks", "tokens", "parents"), (picks, tokens, parents))
    if tokens.dim() != 2:
        raise DartError("tokens must be [B, N]")
    B, N = tokens.shape
    _sizes(B, N)
    _check_tensor(tokens, "tokens", torch.int32)
    _check_tensor(parents, "parents", torch.int32, (B, N))
    _check_tensor(picks, "picks", torch.int32, (B, N + 1))
    if not 0 <= depth <= N:
        raise DartError(f"depth must be 0..{N}, got {depth}")
    scope = _enter(dev, stream)
    try:
        path = torch.empty((B, depth + 1), dtype=torch.int32, device=dev)
        counts = torch.empty(B, dtype=torch.int32, device=dev)
        out = torch.empty((B, depth + 1), dtype=torch.int32, device=dev)
        rc = lib().dart_tree_accept(picks.data_ptr(), tokens.data_ptr(), parents.data_ptr(), B, N, depth,
                                    path.data_ptr(), counts.data_ptr(), out.data_ptr(), _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_tree_accept")
    return {"path": path, "counts": counts, "tokens": out}


def _one_length(lengths):
    if lengths.dim() != 1:
        raise DartError("lengths must be [B]")
    _check_tensor(lengths, "lengths", _torch().int32)
    return lengths.shape[0]


def kv_keep(k_cache, v_cache, pages, lengths, path, counts, *, scores=None, starts=None, device_err=None, stream=None):
    """Moves a path's keys and values up behind one another (dart_kv_keep).

    k_cache, v_cache, pages, lengths as for kv_append (lengths: the tokens in
    the cache before the chunk), the caches written in place; path (int32 [B,
    width], increasing) and counts (int32 [B]) as tree_accept returns them.
    scores (float32 [B, heads, width], from attention_weights) move with their
    positions, in place, and become 0 from the new lengths to the chunk's end,
    which starts (int32 [B + 1], the chunk's) tell: a cache that is ever given to
    kv_evict needs them here (dart_kv_keep_scored).  Returns the new lengths,
    lengths + counts: one call per layer reads the old ones.  device_err (int32
    [>= 1], zeroed by the caller) collects the error bits of what is out of range
    or out of order."""
    if stream is None and k_cache.is_cuda:
        made = _native().keep(k_cache, v_cache, pages, lengths, path, counts, scores, starts, device_err)
        if made is not None:
            return made
    torch = _torch()
    dev = _one_device(("k_cache", "v_cache", "pages", "lengths", "path", "counts", "scores", "starts", "device_err"),
                      (k_cache, v_cache, pages, lengths, path, counts, scores, starts, device_err))
    B = _one_length(lengths)
    c = _cache(k_cache, v_cache, pages, B)
    if path.dim() != 2 or path.shape[0] != B or path.shape[1] < 1:
        raise DartError(f"path must be [{B}, width], width >= 1")
    _check_tensor(path, "path", torch.int32, contiguous=False)
    _check_inner(path, "path")
    width = path.shape[1]
    _sizes(B, width)
    step = path.stride(0) if B > 1 else width
    if step < width:
        raise DartError("the rows of path overlap")
    _check_tensor(counts, "counts", torch.int32, (B,))
    if (scores is None) != (starts is None):
        raise DartError("scores need the chunk's starts, and starts are of use with scores alone")
    if scores is not None:
        s0, s1 = _scores(scores, B, c.heads)
        _check_tensor(starts, "starts", torch.int32, (B + 1,))
    if device_err is not None:
        _check_error_word(device_err)
    name = "dart_kv_keep" if scores is None else "dart_kv_keep_scored"
    scope = _enter(dev, stream)
    try:
        out = torch.empty(B, dtype=torch.int32, device=dev)
        gathered = () if scores is None else (starts.data_ptr(), scores.data_ptr(), s0, s1, scores.shape[2])
        rc = getattr(lib(), name)(C.byref(c), lengths.data_ptr(), path.data_ptr(), step, counts.data_ptr(), B, width,
                                  *gathered, out.data_ptr(), _at(device_err), _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, name)
    return out


# ----------------------------------------------------------------- eviction

def _scores(scores, B, heads):
    """The (sequence, head) strides of float32 scores [B, heads, width]."""
    if scores.dim() != 3 or scores.shape[0] != B or scores.shape[1] != heads:
        raise DartError(f"scores must be [{B}, {heads}, width]")
    _check_tensor(scores, "scores", _torch().float32, contiguous=False)
    _check_inner(scores, "scores")
    width = scores.shape[2]
    _sizes(B, width)
    a, b = scores.stride(0) if B > 1 else heads * width, scores.stride(1) if heads > 1 else width
    low, high = sorted(((a, B), (b, heads)))
    if width and ((heads > 1 and b < width) or (B > 1 and a < width) or
                  (B > 1 and heads > 1 and high[0] < low[0] * (low[1] - 1) + width)):
        raise DartError("the rows of scores overlap")
    return a, b


def attention_weights(q, k_cache, pages, lengths, starts, lse, scores, *, mask=None, scale: float | None = None,
                      device_err=None, stream=None):
    """Adds a chunk's attention weights to what each position has gathered (dart_attention_weights).

    q, k_cache, pages, lengths, starts, mask, scale: as in the tree_attention
    call whose lse (float32 [T, q_heads], from lse=True) is given.  scores:
    float32 [B, heads, width], written in place: each position of a key head
    gains the sum of the weights that the chunk's rows of that head gave it.  A
    row whose lse is not finite adds nothing: set it to +inf to leave a row out.
    Returns scores.  device_err (int32 [>= 1], zeroed by the caller) collects
    error bits."""
    if stream is None and q.is_cuda:
        made = _native().weights(q, k_cache, pages, lengths, starts, lse, scores, mask, scale, device_err)
        if made is not None:
            return made
    torch = _torch()
    dev = _one_device(("q", "k_cache", "pages", "lengths", "starts", "lse", "scores", "mask", "device_err"),
                      (q, k_cache, pages, lengths, starts, lse, scores, mask, device_err))
    B = _sequences(lengths, starts)
    c = _cache(k_cache, k_cache, pages, B)
    if q.dim() != 3:
        raise DartError("q must be [T, q_heads, dim]")
    T, Hq, dim = q.shape
    _sizes(T, Hq)
    q0, q1 = _output(q, "q", T, Hq, c.dim, k_cache.dtype)         # copied in boxes, which an expanded tensor has not
    if Hq < 1 or Hq % c.heads:
        raise DartError(f"{Hq} query heads do not share {c.heads} key heads evenly")
    _check_tensor(lse, "lse", torch.float32, (T, Hq))
    s0, s1 = _scores(scores, B, c.heads)
    N = 0
    if mask is not None:
        if mask.dim() != 3 or mask.shape[0] != B or mask.shape[2] != (mask.shape[1] + 31) // 32:
            raise DartError(f"mask must be [{B}, N, ceil(N / 32)]")
        N = mask.shape[1]
        _sizes(N)
        _check_tensor(mask, "mask", _mask_dtypes())
    if device_err is not None:
        _check_error_word(device_err)
    scope = _enter(dev, stream)
    try:
        rc = lib().dart_attention_weights(q.data_ptr(), q0, q1, Hq, T, B, lengths.data_ptr(), starts.data_ptr(),
                                          _at(mask), N, dim ** -0.5 if scale is None else scale, C.byref(c),
                                          lse.data_ptr(), scores.data_ptr(), s0, s1, scores.shape[2],
                                          _at(device_err), _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_attention_weights")
    return scores


def kv_evict(k_cache, v_cache, pages, lengths, scores, keep: int, *, first: int = 4, last: int = 0, device_err=None,
             stream=None) -> dict:
    """Brings sequences of more than `keep` tokens back to `keep` (dart_kv_evict).

    Per key head the first `first` positions, the last `last` and those between
    with the largest scores (float32 [B, heads, width], from attention_weights)
    stay; their keys, values and scores move up in their order, in place, and
    the scores behind become 0.  Keys keep the rotary positions that they were
    written with: later kv_append calls give offsets that make up for the
    shortened lengths.  Returns lengths (int32 [B], the new ones) and index
    (int32 [B, heads, keep], the old position of each slot, -1 from the length
    on).  device_err as for kv_keep."""
    if stream is None and k_cache.is_cuda:
        made = _native().evict(k_cache, v_cache, pages, lengths, scores, keep, first, last, device_err)
        if made is not None:
            return {"lengths": made[0], "index": made[1]}
    torch = _torch()
    dev = _one_device(("k_cache", "v_cache", "pages", "lengths", "scores", "device_err"),
                      (k_cache, v_cache, pages, lengths, scores, device_err))
    B = _one_length(lengths)
    c = _cache(k_cache, v_cache, pages, B)
    s0, s1 = _scores(scores, B, c.heads)
    _sizes(keep)
    if keep < 1 or first < 0 or last < 0 or first + last > keep:
        raise DartError(f"keep ({keep}) must hold the first {first} and the last {last} positions, and be at least 1")
    if device_err is not None:
        _check_error_word(device_err)
    scope = _enter(dev, stream)
    try:
        index = torch.empty((B, c.heads, keep), dtype=torch.int32, device=dev)
        out = torch.empty(B, dtype=torch.int32, device=dev)
        rc = lib().dart_kv_evict(C.byref(c), lengths.data_ptr(), B, scores.data_ptr(), s0, s1, scores.shape[2], keep,
                                 first, last, index.data_ptr(), out.data_ptr(), _at(device_err), _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_kv_evict")
    return {"lengths": out, "index": index}
