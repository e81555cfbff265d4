// dart_append.cu -- K6: a chunk's keys and values into a paged cache, with the
// norms of query and key heads and the rotary positions in the same pass.
//
// One warp takes four heads of one token at a time, eight lanes a head, two
// 16-byte vectors a lane: the two vectors hold the two elements of each pair
// (half layout), or neighbouring pairs (interleaved), so the turn needs no
// exchange, a norm is one reduction over eight lanes, and the sines and
// cosines, which depend on the token and the lane alone, are computed once and
// serve every head that the warp takes.
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kAppThreads = 128;
constexpr int kBatch = 3;             // quads of heads that a warp has under way

struct AppendParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
  int Hq, Hkv, D, T, B;
  const int32_t* lengths;
  const int32_t* starts;
  const int32_t* offsets;
  const uint64_t* turns;      // nullptr: no turn
  float magnitude;
  int rot, interleaved;
  const void* q_weight;
  const void* k_weight;
  float eps;
  dart_cache_t c;
  int quads, parts;           // groups of four heads; warps per token
  FastDiv by_parts, by_page;
  float inv_dim;
  uint32_t* err;
};

// A 32-bit word of two elements as two fp32 values, and back.
template <typename T> __device__ __forceinline__ uint64_t unpack2(uint32_t w);
template <> __device__ __forceinline__ uint64_t unpack2<__half>(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  const float2 f = __half22float2(h);
  return pair(f.x, f.y);
}
template <> __device__ __forceinline__ uint64_t unpack2<__nv_bfloat16>(uint32_t w) {
  return uint64_t(w << 16) | (uint64_t(w & 0xFFFF0000u) << 32);
}
template <typename T> __device__ __forceinline__ uint32_t pack2(uint64_t x);
template <> __device__ __forceinline__ uint32_t pack2<__half>(uint64_t x) {
  const __half2 h = __floats2half2_rn(low(x), high(x));
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(uint64_t x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(low(x), high(x));
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <typename T> __device__ __forceinline__ void unpack8(uint4 u, uint64_t* x) {
  x[0] = unpack2<T>(u.x);
  x[1] = unpack2<T>(u.y);
  x[2] = unpack2<T>(u.z);
  x[3] = unpack2<T>(u.w);
}
template <typename T> __device__ __forceinline__ uint4 pack8(const uint64_t* x) {
  return make_uint4(pack2<T>(x[0]), pack2<T>(x[1]), pack2<T>(x[2]), pack2<T>(x[3]));
}
__device__ __forceinline__ uint64_t swap2(uint64_t x) { return (x << 32) | (x >> 32); }

// The sequence of token t: the number of entries of starts[1..B] that are <= t
// (B when t lies behind them all).  The 32 lanes probe together.
__device__ __forceinline__ int find_sequence(const int32_t* starts, int B, int t, int lane) {
  int lo = 0, hi = B;                       // the answer lies in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;   // probes starts[i], i in (lo, hi]
    const bool below = i <= hi && starts[i] <= t;
    const int n = __popc(__ballot_sync(kFull, below));
    lo = min(lo + n * step, hi);
    // the next probe was above t (or past hi): the answer is less than one step away
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

template <typename T>
__global__ void __launch_bounds__(kAppThreads)
append_kernel(const AppendParams P) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kAppThreads / 32) + (threadIdx.x >> 5);
  const int t = P.by_parts.div(unit), part = unit - t * P.parts;
  if (t >= P.T) return;

  // this lane's two vectors of a head
  const int sub = lane & 7;
  const int rv = P.rot >> 4;                 // lanes that turn; each holds one vector of either half
  const int nv = P.D >> 3;
  const bool turns = sub < rv;
  int va, vb;
  if (turns) {
    va = P.interleaved ? 2 * sub : sub;
    vb = P.interleaved ? 2 * sub + 1 : sub + rv;
  } else {
    va = 2 * rv + 2 * (sub - rv);
    vb = va + 1;
  }
  const bool has_a = va < nv, has_b = vb < nv;

  // The heads' vectors are asked for first, kBatch quads at a time: everything
  // that follows up to their use (the token's sequence, its page, its angles)
  // waits for memory as well.
  uint4 ua[kBatch], ub[kBatch];
  auto fetch = [&](int first) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int quad = first + i * P.parts, h = 4 * quad + (lane >> 3);
      const T* src = nullptr;
      if (h < P.Hq) src = static_cast<const T*>(P.q) + (long long)t * P.q_ts + (long long)h * P.q_hs;
      else if (h < P.Hq + P.Hkv)
        src = static_cast<const T*>(P.k) + (long long)t * P.k_ts + (long long)(h - P.Hq) * P.k_hs;
      else if (h < P.Hq + 2 * P.Hkv)
        src = static_cast<const T*>(P.v) + (long long)t * P.v_ts + (long long)(h - P.Hq - P.Hkv) * P.v_hs;
      ua[i] = ub[i] = make_uint4(0, 0, 0, 0);
      if (src && has_a) ua[i] = *reinterpret_cast<const uint4*>(src + 8 * va);
      if (src && has_b) ub[i] = *reinterpret_cast<const uint4*>(src + 8 * vb);
    }
  };
  fetch(part);
  uint64_t phase[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) phase[j] = turns ? P.turns[8 * sub + j] : 0ull;

  const int b = find_sequence(P.starts, P.B, t, lane);
  if (b >= P.B) return;
  const int index = t - P.starts[b];
  if (index < 0) return;
  const int len = P.lengths[b];
  const long long slot = (long long)len + index;
  const dart_cache_t& C = P.c;
  bool fits = len >= 0 && slot < (long long)C.table_width * C.page;
  int page = 0, in_page = 0;
  if (fits) {
    const int at = P.by_page.div(int(slot));
    page = C.table[(long long)b * C.table_stride + at];
    in_page = int(slot) - at * C.page;
  }

  uint64_t cs[4], sn[4];                     // of this lane's pairs 2j, 2j + 1
  if (turns) {
    const long long pos = P.offsets ? (long long)len + P.offsets[t] : slot;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float s[2], c[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // the position's phase as a fraction of a turn, exact modulo 2^64; its upper half in half turns
        const uint64_t turned = uint64_t(pos) * phase[2 * j + e];
        sincospif(float(int32_t(uint32_t(turned >> 32))) * 0x1p-31f, &s[e], &c[e]);
      }
      sn[j] = pair(s[0] * P.magnitude, s[1] * P.magnitude);
      cs[j] = pair(c[0] * P.magnitude, c[1] * P.magnitude);
    }
  }
  if (fits) fits = page >= 0 && page < C.pages;
  if (!fits && part == 0 && lane == 0) set_dev_error(P.err, DART_DEVERR_CACHE);

  for (int first = part; first < P.quads; first += kBatch * P.parts) {
    if (first != part) fetch(first);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int quad = first + i * P.parts, h = 4 * quad + (lane >> 3);
      if (quad >= P.quads) break;
      const bool is_q = h < P.Hq, is_k = !is_q && h < P.Hq + P.Hkv, is_v = !is_q && !is_k && h < P.Hq + 2 * P.Hkv;
      T* dst = nullptr;
      const T* weight = nullptr;
      if (is_q) {
        dst = static_cast<T*>(P.out) + (long long)t * P.o_ts + (long long)h * P.o_hs;
        weight = static_cast<const T*>(P.q_weight);
      } else if (is_k) {
        if (fits)
          dst = static_cast<T*>(C.k) + (long long)page * C.k_page_stride + (long long)in_page * C.k_row_stride +
                (long long)(h - P.Hq) * C.k_head_stride;
        weight = static_cast<const T*>(P.k_weight);
      } else if (is_v && fits) {
        dst = static_cast<T*>(C.v) + (long long)page * C.v_page_stride + (long long)in_page * C.v_row_stride +
              (long long)(h - P.Hq - P.Hkv) * C.v_head_stride;
      }
      if ((is_q || is_k) && (weight || P.rot > 0)) {
        uint64_t xa[4], xb[4];
        unpack8<T>(ua[i], xa);
        unpack8<T>(ub[i], xb);
        if (weight) {
          uint64_t ss = mul2(xa[0], xa[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) ss = fma2(xa[j], xa[j], ss);
#pragma unroll
          for (int j = 0; j < 4; ++j) ss = fma2(xb[j], xb[j], ss);
          float sum = low(ss) + high(ss);
#pragma unroll
          for (int s = 1; s < 8; s <<= 1) sum += __shfl_xor_sync(0xFFu << (lane & 24), sum, s);
          const float inv = rsqrtf(fmaf(sum, P.inv_dim, P.eps));
          const uint64_t inv2 = pair(inv, inv);
          uint64_t wa[4], wb[4];
          unpack8<T>(has_a ? *reinterpret_cast<const uint4*>(weight + 8 * va) : make_uint4(0, 0, 0, 0), wa);
          unpack8<T>(has_b ? *reinterpret_cast<const uint4*>(weight + 8 * vb) : make_uint4(0, 0, 0, 0), wb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xa[j] = mul2(xa[j], mul2(inv2, wa[j]));
            xb[j] = mul2(xb[j], mul2(inv2, wb[j]));
          }
        }
        if (turns) {
          if (P.interleaved) {
            // vectors 2 sub, 2 sub + 1 hold pairs 8 sub .. 8 sub + 7: (x, y) -> (x c - y s, y c + x s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t ca = cs[j >> 1], sa = sn[j >> 1], cb = cs[2 + (j >> 1)], sb = sn[2 + (j >> 1)];
              const float c0 = j & 1 ? high(ca) : low(ca), s0 = j & 1 ? high(sa) : low(sa);
              const float c1 = j & 1 ? high(cb) : low(cb), s1 = j & 1 ? high(sb) : low(sb);
              xa[j] = fma2(swap2(xa[j]), pair(-s0, s0), mul2(xa[j], pair(c0, c0)));
              xb[j] = fma2(swap2(xb[j]), pair(-s1, s1), mul2(xb[j], pair(c1, c1)));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint64_t x = xa[j], y = xb[j], minus = sn[j] ^ 0x8000000080000000ull;
              xa[j] = fma2(y, minus, mul2(x, cs[j]));
              xb[j] = fma2(x, sn[j], mul2(y, cs[j]));
            }
          }
        }
        ua[i] = pack8<T>(xa);
        ub[i] = pack8<T>(xb);
      }
      if (dst && has_a) *reinterpret_cast<uint4*>(dst + 8 * va) = ua[i];
      if (dst && has_b) *reinterpret_cast<uint4*>(dst + 8 * vb) = ub[i];
    }
  }
}

bool mult8(long long a, long long b) { return ((a | b) & 7) == 0; }
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int check_cache(const dart_cache_t* c, int B) {
  if (!c || (c->dtype != DART_F16 && c->dtype != DART_BF16)) return DART_ERR_INVALID_ARG;
  if (c->heads < 1 || c->heads > 65535 || c->dim < 8 || c->dim > 128 || c->dim % 8 != 0) return DART_ERR_INVALID_ARG;
  if (c->page < 8 || c->page % 8 != 0 || c->page > (1 << 20) || c->pages < 0 || c->table_width < 0)
    return DART_ERR_INVALID_ARG;
  if ((long long)c->table_width * c->page > (1ll << 30)) return DART_ERR_INVALID_ARG;
  if (c->table_stride < 0 || (B > 1 && c->table_stride < c->table_width)) return DART_ERR_INVALID_ARG;
  const long long st[6] = {c->k_page_stride, c->k_row_stride, c->k_head_stride,
                           c->v_page_stride, c->v_row_stride, c->v_head_stride};
  for (long long s : st)
    if (s < 0 || s % 8 != 0 || s >= (1ll << 39)) return DART_ERR_INVALID_ARG;
  if (c->pages > 0 && (!aligned16(c->k) || !aligned16(c->v))) return DART_ERR_INVALID_ARG;
  if (B > 0 && c->table_width > 0 && !c->table) return DART_ERR_INVALID_ARG;
  return DART_OK;
}

}  // namespace dart

extern "C" int dart_rotary_pack_host(const double* freqs, int count, uint64_t* turns) {
  if (count < 0 || (count > 0 && (!freqs || !turns))) return DART_ERR_INVALID_ARG;
  // 1 / (2 pi) to 192 bits, the most significant word first: the product with a
  // double's 53-bit mantissa keeps far more than the 64 bits wanted, in integers,
  // so every machine gets the same turns
  const uint64_t inv_two_pi[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull,
                                  0x36d8a5664f10e410ull};
  for (int j = 0; j < count; ++j) {
    const double f = freqs[j];
    if (!std::isfinite(f) || std::fabs(f) >= 2147483648.0) return DART_ERR_INVALID_ARG;
    int e = 0;
    const uint64_t m = uint64_t(std::ldexp(std::frexp(std::fabs(f), &e), 53));
    e -= 53;                                   // |f| = m 2^e, e <= -22
    // m / (2 pi) = (word[0] 2^192 + word[1] 2^128 + word[2] 2^64 + word[3]) 2^-192
    uint64_t word[4] = {0, 0, 0, 0};
    unsigned __int128 carry = 0;
    for (int i = 2; i >= 0; --i) {
      carry += (unsigned __int128)m * inv_two_pi[i];
      word[i + 1] = uint64_t(carry);
      carry >>= 64;
    }
    word[0] = uint64_t(carry);
    // times 2^e: the fraction's upper 64 bits lie `down` bits above word[1]'s
    const int down = -e;
    uint64_t t = 0;
    if (down < 128) {
      const unsigned __int128 top = ((unsigned __int128)word[0] << 64) | word[1];
      t = uint64_t(top >> down);
      t += uint64_t(top >> (down - 1)) & 1u;   // to the nearest
    }
    turns[j] = f < 0 ? 0ull - t : t;
  }
  return DART_OK;
}

extern "C" int dart_kv_append(const void* q, int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                              const void* k, int64_t k_token_stride, int64_t k_head_stride,
                              const void* v, int64_t v_token_stride, int64_t v_head_stride,
                              int T, int B, const int32_t* lengths, const int32_t* starts, const int32_t* offsets,
                              const dart_rotary_t* rotary, const void* q_weight, const void* k_weight, float eps,
                              const dart_cache_t* cache, void* out, int64_t out_token_stride,
                              int64_t out_head_stride, uint32_t* device_err, void* stream) {
  using namespace dart;
  if (T < 0 || T > (1 << 26) || B < 0 || q_heads < 0 || q_heads > 65535) return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return DART_ERR_INVALID_ARG;
  if (rotary) {
    if (rotary->reserved != 0 || rotary->rot < 16 || rotary->rot % 16 != 0 || rotary->rot > cache->dim ||
        !std::isfinite(rotary->magnitude) || (rotary->interleaved != 0 && rotary->interleaved != 1) ||
        !rotary->turns)
      return DART_ERR_INVALID_ARG;
  }
  if (T == 0 || B == 0) return DART_OK;
  if (!aligned16(k) || !aligned16(v) || !mult8(k_token_stride, k_head_stride) || !mult8(v_token_stride, v_head_stride))
    return DART_ERR_INVALID_ARG;
  if (q_heads > 0 && (!aligned16(q) || !aligned16(out) || !mult8(q_token_stride, q_head_stride) ||
                      !mult8(out_token_stride, out_head_stride)))
    return DART_ERR_INVALID_ARG;
  if ((q_weight && !aligned16(q_weight)) || (k_weight && !aligned16(k_weight))) return DART_ERR_INVALID_ARG;
  if (!lengths || !starts) return DART_ERR_INVALID_ARG;
  AppendParams P;
  P.q = q; P.k = k; P.v = v; P.out = out;
  P.q_ts = q_token_stride; P.q_hs = q_head_stride;
  P.k_ts = k_token_stride; P.k_hs = k_head_stride;
  P.v_ts = v_token_stride; P.v_hs = v_head_stride;
  P.o_ts = out_token_stride; P.o_hs = out_head_stride;
  P.Hq = q_heads; P.Hkv = cache->heads; P.D = cache->dim; P.T = T; P.B = B;
  P.lengths = lengths; P.starts = starts; P.offsets = offsets;
  P.turns = rotary ? rotary->turns : nullptr;
  P.magnitude = rotary ? rotary->magnitude : 1.f;
  P.rot = rotary ? rotary->rot : 0;
  P.interleaved = rotary ? rotary->interleaved : 0;
  P.q_weight = q_weight; P.k_weight = k_weight; P.eps = eps;
  P.c = *cache;
  P.err = device_err;
  P.quads = (q_heads + 2 * cache->heads + 3) / 4;
  // A warp takes one batch of quads when tokens are few, then several, so that
  // the angles are computed once for as many heads as the number of warps allows.
  const long long want = 152ll * 32;
  long long parts = (want + T - 1) / T;
  P.parts = int(parts < 1 ? 1 : parts > P.quads ? P.quads : parts);
  P.by_parts = fast_div(uint32_t(P.parts));
  P.by_page = fast_div(uint32_t(cache->page));
  P.inv_dim = 1.f / float(cache->dim);
  const long long warps = (long long)T * P.parts;
  const unsigned grid = unsigned((warps + kAppThreads / 32 - 1) / (kAppThreads / 32));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->dtype == DART_F16) append_kernel<__half><<<grid, kAppThreads, 0, s>>>(P);
  else append_kernel<__nv_bfloat16><<<grid, kAppThreads, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
