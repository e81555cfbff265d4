"""The steps around a draft tree: logit adjustment, cache append, tree attention.

Bindings of dart_logits_adjust, dart_kv_append and dart_tree_attention
(include/darttree.h); the package exports the public names.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import importlib.util
import math
import os
import warnings

import numpy as np

from . import (DTYPE_CODES, DartError, _check, _check_error_word, _check_tensor, _check_workspace, _device_of,
               _mask_dtypes, _on_device, _row_stride, _stream_ptr, _torch, lib)
from ._build import native_path


_codes = functools.cache(DTYPE_CODES)


class _Adjust(C.Structure):
    _fields_ = [("history", C.c_void_p), ("history_stride", C.c_int64), ("history_width", C.c_int32),
                ("bias_count", C.c_int32), ("history_len", C.c_void_p), ("repetition", C.c_void_p),
                ("presence", C.c_void_p), ("frequency", C.c_void_p), ("bias_ids", C.c_void_p),
                ("bias_vals", C.c_void_p), ("allowed", C.c_void_p), ("allowed_seq_stride", C.c_int64),
                ("allowed_row_stride", C.c_int64), ("tokens", C.c_void_p), ("mask", C.c_void_p),
                ("N", C.c_int32), ("reserved", C.c_int32)]


class _Cache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p),
                *((f"{x}_{y}_stride", C.c_int64) for x in "kv" for y in ("page", "row", "head")),
                ("table", C.c_void_p), ("table_stride", C.c_int64), ("table_width", C.c_int32), ("pages", C.c_int32),
                ("page", C.c_int32), ("heads", C.c_int32), ("dim", C.c_int32), ("dtype", C.c_int32)]


class _Rotary(C.Structure):
    _fields_ = [("turns", C.c_void_p), ("magnitude", C.c_float), ("rot", C.c_int32), ("interleaved", C.c_int32),
                ("reserved", C.c_int32)]


def declare(L):
    P, i32, i64, f32, sz = C.c_void_p, C.c_int, C.c_int64, C.c_float, C.c_size_t
    L.dart_logits_adjust.argtypes = [P, i32, i32, i32, i64, i32, C.POINTER(_Adjust), P, i64, P]
    L.dart_logits_adjust.restype = i32
    L.dart_rotary_pack_host.argtypes = [P, i32, P]
    L.dart_rotary_pack_host.restype = i32
    L.dart_kv_append.argtypes = [P, i64, i64, i32, P, i64, i64, P, i64, i64, i32, i32, P, P, P, C.POINTER(_Rotary),
                                 P, P, f32, C.POINTER(_Cache), P, i64, i64, P, P]
    L.dart_kv_append.restype = i32
    L.dart_attention_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.dart_attention_workspace_bytes.restype = sz
    L.dart_tree_attention.argtypes = [P, i64, i64, i32, i32, i32, P, P, P, i32, f32, C.POINTER(_Cache), P, i64, i64,
                                      P, P, sz, P]
    L.dart_tree_attention.restype = i32


# A call's host work is a good part of a small call's time: _steps_native makes
# the usual calls, and returns None for those that it leaves to the code here (a
# stream is given, the tensors are not on the current device, something is empty
# or wrong), before it has called the library.  The checks here decide on plain
# integers and only a failing one looks for its words.  Without the module every
# call is made by the code here.

_native = None


class _LeaveAll:
    """In the module's place where there is none: every call goes the binding's way."""

    @staticmethod
    def adjust(*args):
        return None

    append = attend = sample = accept = keep = weights = evict = bind_verified = adjust


def _load_native():
    global _native
    L = lib()
    _torch()                                   # its libraries first
    path = native_path()
    try:
        if path is None or not os.path.exists(path):
            raise ImportError(f"{path} is missing: run draft_tree_construction_gb300.build()")
        spec = importlib.util.spec_from_file_location("_steps_native", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        _native = _LeaveAll
        warnings.warn(f"calls of the steps around a tree take some microseconds longer: {e}", RuntimeWarning,
                      stacklevel=3)
        return _native
    module.bind(*(C.cast(f, C.c_void_p).value for f in (L.dart_logits_adjust, L.dart_kv_append, L.dart_tree_attention,
                                                        L.dart_attention_workspace_bytes)), _check)
    _native = module
    return module


@contextlib.contextmanager
def _elsewhere(dev, stream):
    with _on_device(dev):
        _stream_ptr(stream, dev)
        with _torch().cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            yield


def _enter(dev, stream):
    """Makes the tensors' device current, and the stream that the call launches
    on, so that what the call allocates and clears itself is ordered with its
    kernels.  Returns what _leave takes; None where nothing has to change."""
    if stream is None and dev.index == _torch().cuda.current_device():
        return None
    scope = _elsewhere(dev, stream)
    scope.__enter__()
    return scope


def _leave(scope):
    if scope is not None:
        scope.__exit__(None, None, None)


def _stream(stream, dev):
    """The stream's handle as an integer (the current one's without a stream)."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(dev.index)
    return stream.cuda_stream


def _at(t):
    return None if t is None else t.data_ptr()


def _one_device(names, tensors):
    """The one CUDA device of the tensors that are given."""
    index = tensors[0].get_device()
    if index >= 0:
        for t in tensors:
            if t is not None and t.get_device() != index:
                break
        else:
            return tensors[0].device
    return _device_of(*zip(names, tensors))


def _check_inner(t, name):
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise DartError(f"{name} must have unit stride in its last dimension")


# --------------------------------------------------------- logit adjustment

def adjust_logits(logits, *, history=None, lengths=None, repetition=None, presence=None, frequency=None, bias=None,
                  allowed=None, tokens=None, mask=None, out=None, stream=None):
    """Penalties for repeated tokens, biases and a grammar mask (dart_logits_adjust).

    logits: CUDA [B, R, V] float32/float16/bfloat16, rows evenly spaced (a view
    of a padded vocabulary serves): draft rows, or the verified rows of a tree.
    history: int32 [B, H], of which lengths (int32 [B]) entries count; ids
    outside [0, V) do not.  repetition, presence, frequency: float32 [B], all
    over that one history: repetition over a prompt and what was generated, the
    others over what was generated alone, take two calls (the second in place).
    bias: (ids int32 [B, K], values float32 [B, K]).  allowed: packed bits,
    int32 (or uint32) [B, ceil(V/32)] or [B, R, ceil(V/32)].  tokens (int32
    [B, N]) and mask (int32 [B, N, ceil(N/32)]) of a tree, as tree_build
    returns them, let row R - N + i count the tokens on node i's path too; R
    is N or N + 1.  Returns the adjusted logits: out, which may be logits
    itself, or a new [B, R, V] tensor with evenly spaced rows."""
    ids, vals = bias if bias is not None else (None, None)
    if stream is None and logits.is_cuda:
        made = (_native or _load_native()).adjust(logits, history, lengths, repetition, presence, frequency, ids, vals,
                                                  allowed, tokens, mask, out)
        if made is not None:
            return made
    torch = _torch()
    dev = _one_device(("logits", "history", "lengths", "repetition", "presence", "frequency", "bias ids",
                       "bias values", "allowed", "tokens", "mask", "out"),
                      (logits, history, lengths, repetition, presence, frequency, ids, vals, allowed, tokens, mask,
                       out))
    code = _codes().get(logits.dtype)
    if code is None or logits.dim() != 3:
        raise DartError("logits must be [B, R, V] float32, float16 or bfloat16")
    B, R, V = logits.shape
    if V < 1:
        raise DartError("logits must have at least one token")
    stride = V if logits.is_contiguous() else _row_stride(logits)
    a = _Adjust()
    if history is not None:
        if history.dim() != 2 or history.shape[0] != B:
            raise DartError(f"history must be [{B}, H]")
        _check_tensor(history, "history", torch.int32, contiguous=False)
        _check_inner(history, "history")
        a.history, a.history_width = history.data_ptr(), history.shape[1]
        a.history_stride = history.stride(0) if B > 1 else history.shape[1]
        if B > 1 and a.history_stride < history.shape[1]:
            raise DartError("history rows overlap")
    elif lengths is not None:
        raise DartError("lengths are given without a history")
    if lengths is not None:
        _check_tensor(lengths, "lengths", torch.int32, (B,))
        a.history_len = lengths.data_ptr()
    if repetition is not None:
        _check_tensor(repetition, "repetition", torch.float32, (B,))
        a.repetition = repetition.data_ptr()
    if presence is not None:
        _check_tensor(presence, "presence", torch.float32, (B,))
        a.presence = presence.data_ptr()
    if frequency is not None:
        _check_tensor(frequency, "frequency", torch.float32, (B,))
        a.frequency = frequency.data_ptr()
    if ids is not None:
        if vals is None or ids.dim() != 2 or ids.shape[0] != B:
            raise DartError(f"bias must be (ids [{B}, K], values [{B}, K])")
        _check_tensor(ids, "bias ids", torch.int32)
        _check_tensor(vals, "bias values", torch.float32, tuple(ids.shape))
        a.bias_ids, a.bias_vals, a.bias_count = ids.data_ptr(), vals.data_ptr(), ids.shape[1]
    if allowed is not None:
        words = (V + 31) // 32
        if tuple(allowed.shape) not in ((B, words), (B, R, words)):
            raise DartError(f"allowed must be [{B}, {words}] or [{B}, {R}, {words}], got {tuple(allowed.shape)}")
        _check_tensor(allowed, "allowed", _mask_dtypes(), contiguous=False)
        _check_inner(allowed, "allowed")
        a.allowed, a.allowed_seq_stride = allowed.data_ptr(), allowed.stride(0) if B > 1 else 0
        a.allowed_row_stride = allowed.stride(1) if allowed.dim() == 3 and R > 1 else 0
    if (tokens is None) != (mask is None):
        raise DartError("a tree needs both its tokens and its mask")
    if tokens is not None:
        if tokens.dim() != 2 or tokens.shape[0] != B:
            raise DartError(f"tokens must be [{B}, N]")
        N = tokens.shape[1]
        _check_tensor(tokens, "tokens", torch.int32)
        _check_tensor(mask, "mask", _mask_dtypes(), (B, N, (N + 31) // 32))
        if R not in (N, N + 1):
            raise DartError(f"a tree of {N} nodes needs {N} or {N + 1} rows of logits, got {R}")
        a.tokens, a.mask, a.N = tokens.data_ptr(), mask.data_ptr(), N
    out_stride = 0
    if out is not None:
        _check_tensor(out, "out", logits.dtype, (B, R, V), contiguous=False)
        out_stride = _row_stride(out)
        if out.data_ptr() == logits.data_ptr() and out_stride != stride and B * R > 1:
            raise DartError("out shares its first element with logits, but not its rows")
    scope = _enter(dev, stream)
    try:
        if out is None:
            # rows that keep the input's alignment take whole vectors from end to end
            out_stride = V + (stride - V) % (16 // logits.element_size())
            out = torch.empty((B, R, out_stride), dtype=logits.dtype, device=dev)
            if out_stride != V:
                out = out[..., :V]
        rc = lib().dart_logits_adjust(logits.data_ptr(), B, R, V, stride, code, C.byref(a), out.data_ptr(),
                                      out_stride, _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_logits_adjust")
    return out


# ------------------------------------------------------------- paged caches

def _cache(k_cache, v_cache, pages, B):
    """The descriptor of caches [P, page, heads, dim] with a page table [B, width]."""
    torch = _torch()
    shape, dt = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise DartError("k_cache and v_cache must both be [pages, page, heads, dim]")
    if dt not in (torch.float16, torch.bfloat16) or v_cache.dtype != dt:
        raise DartError("k_cache and v_cache must both be float16 or bfloat16")
    table, (width, step) = pages.shape, (pages.shape[-1], pages.stride(0) if pages.dim() == 2 else 0)
    if len(table) != 2 or table[0] != B:
        raise DartError(f"pages must be [{B}, width]")
    if pages.dtype != torch.int32:
        _check_tensor(pages, "pages", torch.int32, contiguous=False)
    if width > 1 and pages.stride(1) != 1:
        raise DartError("pages must have unit stride in its last dimension")
    if B <= 1:
        step = width
    elif step < width:
        raise DartError("the rows of pages overlap")
    count, page, heads, dim = shape
    if (width | count | page | heads) >> 31:       # the descriptor holds them in 32 bits
        raise DartError(f"{max(width, count, page, heads)} is more than a cache can have of anything")
    if page < 8 or page & 7:
        raise DartError(f"pages must hold a multiple of 8 positions, got {page}")
    if not 8 <= dim <= 128 or dim & 7:
        raise DartError(f"heads must have a multiple of 8 elements, 8 to 128, got {dim}")
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if k3 != 1 or v3 != 1:
        raise DartError("k_cache and v_cache must have unit stride in their last dimension")
    if count <= 1:                  # a dimension of one is never stepped along
        k0 = v0 = 8
    if heads == 1:
        k2 = v2 = 8
    at, vat = k_cache.data_ptr(), v_cache.data_ptr()
    if (k0 | k1 | k2 | v0 | v1 | v2) & 7 or (at | vat) & 15:
        raise DartError("k_cache and v_cache must be 16-byte aligned, with strides of multiples of 8 elements")
    if not (k0 and k1 and k2 and v0 and v1 and v2):
        # memory shared between elements (an expanded tensor) cannot be written
        raise DartError("k_cache and v_cache must not be expanded tensors")
    return _Cache(at, vat, k0, k1, k2, v0, v1, v2, pages.data_ptr(), step, width, count, page, heads, dim,
                  _codes()[dt])


def _heads(t, name, T, heads, dim, dtype):
    """A [T, heads, dim] tensor of vectors: its (token, head) strides."""
    st = t.stride()
    if t.dtype == dtype and t.shape == (T, heads, dim) and st[2] == 1:
        a, b = st[0] if T > 1 else 0, st[1] if heads > 1 else 0
        if not ((a | b) & 7 or t.data_ptr() & 15):
            return a, b
    _check_tensor(t, name, dtype, (T, heads, dim), contiguous=False)
    _check_inner(t, name)
    raise DartError(f"{name} must be 16-byte aligned, with strides of multiples of 8 elements")


def _output(t, name, T, heads, dim, dtype):
    """_heads of a tensor that is written: its elements share no memory."""
    a, b = _heads(t, name, T, heads, dim, dtype)
    if (a == 0 and T > 1) or (b == 0 and heads > 1):
        raise DartError(f"{name} must not be an expanded tensor")
    return a, b


def _sequences(lengths, starts):
    torch = _torch()
    if lengths.dim() != 1:
        raise DartError("lengths must be [B]")
    B = lengths.shape[0]
    if lengths.dtype != torch.int32 or not lengths.is_contiguous():
        _check_tensor(lengths, "lengths", torch.int32)
    if starts.dtype != torch.int32 or starts.shape != (B + 1,) or not starts.is_contiguous():
        _check_tensor(starts, "starts", torch.int32, (B + 1,))
    return B


class Rotary:
    """Rotary positions for kv_append: pair j of a head turns by position * freqs[j].

    freqs: rot / 2 radians per position (float64; see rotary_frequencies), rot
    the elements of each head that turn, the rest staying as they are.
    magnitude scales the turned elements.  interleaved: pairs (2j, 2j + 1)
    instead of (j, j + rot / 2)."""

    def __init__(self, freqs, magnitude: float = 1.0, interleaved: bool = False, device="cuda"):
        freqs = np.ascontiguousarray(freqs, dtype=np.float64).reshape(-1)
        if freqs.size < 8 or freqs.size % 8 or freqs.size > 64:
            raise DartError("freqs must hold 8, 16, .. 64 values (rot / 2, rot a multiple of 16)")
        if not math.isfinite(magnitude):
            raise DartError("magnitude must be finite")
        turns = np.empty(freqs.size, dtype=np.uint64)
        _check(lib().dart_rotary_pack_host(freqs.ctypes.data_as(C.c_void_p), freqs.size,
                                           turns.ctypes.data_as(C.c_void_p)), "dart_rotary_pack_host")
        self.freqs, self.magnitude, self.interleaved = freqs, float(magnitude), bool(interleaved)
        self.rot = 2 * freqs.size
        self.turns = _torch().from_numpy(turns.view(np.int64)).to(device)
        self.desc = _Rotary(self.turns.data_ptr(), self.magnitude, self.rot, int(self.interleaved), 0)
        self.address = C.addressof(self.desc)


def rotary_frequencies(rot: int, base: float = 10000.0, factor: float = 1.0, original: int | None = None,
                       fast: float = 32.0, slow: float = 1.0):
    """(freqs float64 [rot / 2], magnitude) of rotary positions: base^(-2j / rot).

    factor > 1 stretches them for contexts that are `factor` times longer:
    without `original` every frequency is divided by factor (magnitude 1); with
    it (the length that the model was trained on), a pair that turns more than
    `fast` times within `original` positions keeps its frequency, one that turns
    less than `slow` times is divided by factor, those between are blended
    linearly in their number of turns, and the magnitude is 0.1 ln(factor) + 1.
    Many models are run with another ramp instead: linear in the pair's index
    j between the pairs that turn `fast` and `slow` times, those two rounded to
    whole pairs.  Its frequencies differ between the two ends; for such a model
    give Rotary the frequencies of its own ramp."""
    if rot < 2 or rot % 2 or not base > 0 or not factor >= 1:
        raise DartError("rot must be even, base > 0 and factor >= 1")
    f = float(base) ** (-np.arange(rot // 2, dtype=np.float64) / (rot // 2))
    if factor == 1.0 or original is None:
        return f / factor, 1.0
    if not fast > slow:
        raise DartError("fast must exceed slow")
    keep = np.clip((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


def kv_append(q, k, v, k_cache, v_cache, pages, lengths, starts, *, rotary: Rotary | None = None, offsets=None,
              q_weight=None, k_weight=None, eps: float = 1e-6, out=None, device_err=None, stream=None):
    """Appends a chunk's keys and values to a paged cache (dart_kv_append).

    q: CUDA [T, q_heads, dim] or None; k, v: [T, heads, dim] (views of one
    projection's output serve); k_cache, v_cache: [pages, page, heads, dim],
    float16 or bfloat16 like q, k and v, written in place; pages: int32 [B,
    width], the page of each sequence's positions; lengths: int32 [B] tokens in
    the cache before the chunk; starts: int32 [B + 1], sequence b's tokens being
    rows starts[b] .. starts[b + 1] (rows outside are left alone).  q_weight,
    k_weight ([dim]) apply the norm of each head, rotary the turn by position
    lengths[b] + index in the chunk, or lengths[b] + offsets[row] (int32 [T]; a
    tree's nodes: the root's offset + tree_build's pos).  Returns the finished
    queries: out, which may be q itself, or a new tensor whose rows outside
    every sequence are unset (None without q).  device_err (int32 [>= 1], zeroed
    by the caller) collects the error bits of tokens that do not fit in their
    pages."""
    if stream is None and k.is_cuda:
        turns, address = (rotary.turns, rotary.address) if rotary is not None else (None, 0)
        made = (_native or _load_native()).append(q, k, v, k_cache, v_cache, pages, lengths, starts, turns, address,
                                                  offsets, q_weight, k_weight, eps, out, device_err)
        if made is not None:
            return made
    torch = _torch()
    dev = _one_device(("k", "v", "q", "k_cache", "v_cache", "pages", "lengths", "starts", "rotary", "offsets",
                       "q_weight", "k_weight", "out", "device_err"),
                      (k, v, q, k_cache, v_cache, pages, lengths, starts,
                       rotary.turns if rotary is not None else None, offsets, q_weight, k_weight, out, device_err))
    B = _sequences(lengths, starts)
    c = _cache(k_cache, v_cache, pages, B)
    if k.dim() != 3:
        raise DartError("k must be [T, heads, dim]")
    T, dt, dim = k.shape[0], k_cache.dtype, c.dim
    k0, k1 = _heads(k, "k", T, c.heads, dim, dt)
    v0, v1 = _heads(v, "v", T, c.heads, dim, dt)
    Hq = q0 = q1 = o0 = o1 = 0
    if q is not None:
        if q.dim() != 3:
            raise DartError("q must be [T, q_heads, dim]")
        Hq = q.shape[1]
        q0, q1 = _heads(q, "q", T, Hq, dim, dt)
        if out is not None:
            o0, o1 = _output(out, "out", T, Hq, dim, dt)
            if out.data_ptr() == q.data_ptr() and (o0, o1) != (q0, q1):
                raise DartError("out shares its first element with q, but not its strides")
    elif out is not None or q_weight is not None:
        raise DartError("out or q_weight is given without q")
    if offsets is not None:
        _check_tensor(offsets, "offsets", torch.int32, (T,))
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None and (t.dtype != dt or t.shape != (dim,) or t.stride(0) != 1):
            _check_tensor(t, name, dt, (dim,))
    if rotary is not None and rotary.rot > dim:
        raise DartError(f"rotary turns {rotary.rot} elements of heads of {dim}")
    if device_err is not None:
        _check_error_word(device_err)
    scope = _enter(dev, stream)
    try:
        if q is not None and out is None:
            out = torch.empty((T, Hq, dim), dtype=dt, device=dev)
            o0, o1 = Hq * dim, dim
        rc = lib().dart_kv_append(_at(q), q0, q1, Hq, k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, T, B,
                                  lengths.data_ptr(), starts.data_ptr(), _at(offsets),
                                  C.byref(rotary.desc) if rotary is not None else None, _at(q_weight), _at(k_weight),
                                  eps, C.byref(c), _at(out), o0, o1, _at(device_err), _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_kv_append")
    return out


# ------------------------------------------------------------ tree attention

def attention_workspace_bytes(T: int, B: int, q_heads: int, heads: int, dim: int) -> int:
    return lib().dart_attention_workspace_bytes(T, B, q_heads, heads, dim)


def tree_attention(q, k_cache, v_cache, pages, lengths, starts, *, mask=None, scale: float | None = None, out=None,
                   lse: bool = False, workspace=None, stream=None) -> dict:
    """Attention of a chunk over the paged cache that holds it (dart_tree_attention).

    q: CUDA [T, q_heads, dim] float16 or bfloat16 like the caches (as kv_append
    returns it); k_cache, v_cache, pages, lengths, starts as for kv_append,
    which has written the chunk's own keys and values.  Without a mask every
    token sees the positions up to its own.  mask (int32 [B, N, ceil(N/32)], as
    tree_build returns it) makes the last N tokens of each chunk a tree, each
    node seeing the context, the tokens before the tree and its own path.
    scale defaults to 1 / sqrt(dim).  Returns out [T, q_heads, dim] (a new
    tensor's rows outside every sequence are unset), lse (float32 [T, q_heads]
    with lse=True, else None) and the workspace, whose error bits device_error
    reads.  A workspace is reused by calls in order on one stream; calls that
    may overlap need one each."""
    if stream is None and q.is_cuda:
        made = (_native or _load_native()).attend(q, k_cache, v_cache, pages, lengths, starts, mask, scale, out, lse,
                                                  workspace)
        if made is not None:
            return {"out": made[0], "lse": made[1], "workspace": made[2]}
    torch = _torch()
    dev = _one_device(("q", "k_cache", "v_cache", "pages", "lengths", "starts", "mask", "out", "workspace"),
                      (q, k_cache, v_cache, pages, lengths, starts, mask, out, workspace))
    B = _sequences(lengths, starts)
    c = _cache(k_cache, v_cache, pages, B)
    if q.dim() != 3:
        raise DartError("q must be [T, q_heads, dim]")
    T, Hq, dim = q.shape
    dt, heads = k_cache.dtype, c.heads
    q0, q1 = _heads(q, "q", T, Hq, c.dim, dt)
    if Hq < 1 or Hq % heads:
        raise DartError(f"{Hq} query heads do not share {heads} key heads evenly")
    N = 0
    if mask is not None:
        if mask.dim() != 3 or mask.shape[0] != B or mask.shape[2] != (mask.shape[1] + 31) // 32:
            raise DartError(f"mask must be [{B}, N, ceil(N / 32)]")
        N = mask.shape[1]
        _check_tensor(mask, "mask", _mask_dtypes())
    o0 = o1 = 0
    if out is not None:
        o0, o1 = _output(out, "out", T, Hq, dim, dt)
        if out.numel() and out.data_ptr() == q.data_ptr():
            raise DartError("out must not be q")
    L = lib()
    need = L.dart_attention_workspace_bytes(T, B, Hq, heads, dim)
    room = 0
    if workspace is not None:
        room = workspace.numel() * workspace.element_size()
        if room < need or not workspace.is_contiguous():
            _check_workspace(workspace, need)
    sums = None
    scope = _enter(dev, stream)
    try:
        if out is None:
            out = torch.empty((T, Hq, dim), dtype=dt, device=dev)
            o0, o1 = Hq * dim, dim
        if workspace is None:
            workspace, room = torch.empty(need, dtype=torch.uint8, device=dev), need
            workspace[:256].zero_()
        if lse:
            sums = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        rc = L.dart_tree_attention(q.data_ptr(), q0, q1, Hq, T, B, lengths.data_ptr(), starts.data_ptr(), _at(mask), N,
                                   dim ** -0.5 if scale is None else scale, C.byref(c), out.data_ptr(), o0, o1,
                                   _at(sums), workspace.data_ptr(), room, _stream(stream, dev))
    finally:
        _leave(scope)
    if rc:
        _check(rc, "dart_tree_attention")
    return {"out": out, "lse": sums, "workspace": workspace}
