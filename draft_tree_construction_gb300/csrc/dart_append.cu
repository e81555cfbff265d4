// dart_append.cu -- K6: a chunk's keys and values into a paged cache, with the
// norms of query and key heads and the rotary positions in the same pass.
//
// Mathematics: x^ = w x / sqrt(mean(x^2) + eps);  a pair (x, y) at position p turns
// to (x c - y s, y c + x s), c + i s = m e^(i p f);  fp32, rounded once.
//
// What bounds it: memory, q, k and v read once and written once; then the
// instructions (60% of the issue slots), the lookups of a token's sequence, page
// and position (four loads, one after the other) being hidden behind the heads'.
// One warp takes four heads of one token at a time, eight lanes a head, two
// 16-byte vectors a lane: a lane holds both elements of each of its pairs, so
// the turn needs no exchange, a norm is one reduction over eight lanes, and the
// sines and cosines, which depend on the token alone, are computed once (two
// pairs a lane, then exchanged) and serve every head that the warp takes.  The
// angle is kept in 2^-64 turns, in integers: exact at any position.
//
// Measured (GB300, kernel alone, 32 + 8 + 8 heads of 128):
//   64 trees of 79 rows, norms and half layout, 16-token pages   25 us, 5.0 TB/s
//   8191 tokens, 64 of 128 elements turned, interleaved         34.4 us, 5.9 TB/s
//   one token                                                    3.5 us
// Each lane computing its eight sines itself, and registers in place of the
// ring, took 48, 35 and 4.1 us.
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kAppThreads = 128;
constexpr int kAhead = 5;             // quads of heads that a warp has under way
constexpr int kQuadBytes = 1024;      // two vectors a lane
constexpr int kRingBytes = kAppThreads / 32 * kAhead * kQuadBytes;

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
  int q_quads, k_quads, quads, parts;   // groups of four heads: of q, of k (and v), all; warps per token
  FastDiv by_parts, by_page, by_share;  // by_share: T / B, if B sequences of one length would fill T (else d = 0)
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

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppThreads, 5)
append_kernel(const AppendParams P) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * (kAppThreads / 32) + (threadIdx.x >> 5);
  const int t = P.by_parts.div(unit), part = unit - t * P.parts;
  if (t >= P.T) return;

  // This lane's two vectors of a head; eight lanes' vectors lie side by side.
  // Half layout: the rv lanes that turn hold the two vectors of a pair each, the
  // others what stays.  Interleaved: a pair lies within a vector, so any two do.
  const int sub = lane & 7;
  const int rv = P.rot >> 4, nv = P.D >> 3;
  int va = sub, vb = sub + 8;
  bool turn_a, turn_b;
  if (INTERLEAVED) {
    turn_a = va < 2 * rv;
    turn_b = vb < 2 * rv;
  } else {
    turn_a = turn_b = sub < rv;
    if (turn_a) vb = sub + rv;
    else va = sub + rv, vb = va + 8 - rv;
  }
  const bool has_a = va < nv, has_b = vb < nv;

  // The quads of the queries, then of the keys, then of the values; this warp's are part, part + parts, ...
  struct Segment { const T* src; long long hs; int first, end, heads; };
  auto segment = [&](int kind) {
    Segment g;
    if (kind == 0) {
      g = Segment{static_cast<const T*>(P.q) + (long long)t * P.q_ts, P.q_hs, 0, P.q_quads, P.Hq};
    } else if (kind == 1) {
      g = Segment{static_cast<const T*>(P.k) + (long long)t * P.k_ts, P.k_hs, P.q_quads, P.q_quads + P.k_quads, P.Hkv};
    } else {
      g = Segment{static_cast<const T*>(P.v) + (long long)t * P.v_ts, P.v_hs, P.q_quads + P.k_quads, P.quads, P.Hkv};
    }
    return g;
  };
  // The heads' vectors are asked for first, kAhead quads of them: everything
  // that follows up to their use (the token's sequence, its page, its angles)
  // waits for memory as well.  They arrive in shared memory, each lane reading
  // back what it asked for.
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned char* ring = smem + (threadIdx.x >> 5) * (kAhead * kQuadBytes) + 16 * lane;
  int asked = part, ask_end = 0, ask_heads = 0, ask_h = 0, into = 0;    // the next quad to ask for, its place
  const T* ask_at = nullptr;
  long long ask_step = 0;
  auto ask = [&]() {
    if (asked < P.quads) {
      if (asked >= ask_end) {                // a new segment
        const Segment g = segment(asked < P.q_quads ? 0 : asked < P.q_quads + P.k_quads ? 1 : 2);
        ask_end = g.end;
        ask_heads = g.heads;
        ask_h = 4 * (asked - g.first) + (lane >> 3);
        ask_at = g.src + (long long)ask_h * g.hs;
        ask_step = 4ll * P.parts * g.hs;
      }
      cp_async16(ring + into, ask_at + 8 * va, has_a && ask_h < ask_heads);
      cp_async16(ring + into + 512, ask_at + 8 * vb, has_b && ask_h < ask_heads);
      asked += P.parts;
      ask_h += 4 * P.parts;
      ask_at += ask_step;
    }
    cp_async_commit();
    into = into + kQuadBytes < kAhead * kQuadBytes ? into + kQuadBytes : 0;
  };
#pragma unroll 1
  for (int i = 0; i < kAhead - 1; ++i) ask();
  int quad = part, place = 0;
  const int kind0 = quad < P.q_quads ? 0 : quad < P.q_quads + P.k_quads ? 1 : 2;
  const bool my_pair = 4 * lane < P.rot;     // pairs 2 lane and 2 lane + 1 are this lane's to compute
  const uint64_t turn0 = my_pair ? P.turns[2 * lane] : 0ull, turn1 = my_pair ? P.turns[2 * lane + 1] : 0ull;

  const int off = P.offsets ? P.offsets[t] : 0;
  // chunks of one size (a tree per sequence, a token per sequence) are found without a search
  int b = P.by_share.d ? P.by_share.div(t) : 0;
  int start = P.starts[b], end = P.starts[b + 1], len = P.lengths[b];
  if (t < start || t >= end) {
    b = find_sequence(P.starts, P.B, t, lane);
    if (b < P.B) {
      start = P.starts[b];
      len = P.lengths[b];
    }
  }
  const int index = t - start;
  if (b >= P.B || index < 0) {      // a row of no sequence
    // the copies asked for must have landed before the CTA gives its shared memory up
    cp_async_wait<0>();
    return;
  }
  const long long slot = (long long)len + index;
  const dart_cache_t& C = P.c;
  bool fits = len >= 0 && slot < (long long)C.table_width * C.page;
  int page = 0, in_page = 0;
  if (fits) {
    const int at = P.by_page.div(int(slot));
    page = C.table[(long long)b * C.table_stride + at];
    in_page = int(slot) - at * C.page;
  }

  uint64_t cs[4], sn[4];                     // of this lane's pairs, two at a time (see `from`)
  if (P.rot > 0) {
    const long long pos = P.offsets ? (long long)len + off : slot;
    float s[2], c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // the position's phase as a fraction of a turn, exact modulo 2^64; its upper half in half turns
      const uint64_t turned = uint64_t(pos) * (e ? turn1 : turn0);
      sincospif(float(int32_t(uint32_t(turned >> 32))) * 0x1p-31f, &s[e], &c[e]);
      s[e] *= P.magnitude;
      c[e] *= P.magnitude;
    }
    const uint64_t cc = pair(c[0], c[1]), ss = pair(s[0], s[1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // half layout: pairs 8 sub + 2 j and the next; interleaved: pairs 4 va + 2 j for j < 2, then 4 vb + 2 (j - 2)
      const int from = INTERLEAVED ? (j < 2 ? 2 * va + j : 2 * vb + j - 2) & 31 : (4 * sub + j) & 31;
      cs[j] = __shfl_sync(kFull, cc, from);
      sn[j] = __shfl_sync(kFull, ss, from);
    }
  }
  if (fits) fits = page >= 0 && page < C.pages;
  if (!fits && part == 0 && lane == 0) set_dev_error(P.err, DART_DEVERR_CACHE);

  for (int kind = kind0; kind < 3; ++kind) {
    const Segment g = segment(kind);
    if (quad >= g.end) continue;
    T* dst = nullptr;
    long long dst_hs = 0;
    const T* weight = nullptr;
    if (kind == 0) {
      dst = static_cast<T*>(P.out) + (long long)t * P.o_ts;
      dst_hs = P.o_hs;
      weight = static_cast<const T*>(P.q_weight);
    } else if (kind == 1) {
      dst = static_cast<T*>(C.k) + (long long)page * C.k_page_stride + (long long)in_page * C.k_row_stride;
      dst_hs = C.k_head_stride;
      weight = static_cast<const T*>(P.k_weight);
    } else {
      dst = static_cast<T*>(C.v) + (long long)page * C.v_page_stride + (long long)in_page * C.v_row_stride;
      dst_hs = C.v_head_stride;
    }
    const bool writes = kind == 0 || fits;
    const bool works = kind < 2 && (weight || P.rot > 0);
    // The norm's weight and the turn in one pair of factors: an element is
    //   inv * (x * w cos -+ y * w' sin),  y and w' being its partner and its partner's weight
    uint64_t ka[4], la[4], kb[4], lb[4];
    if (works) {
      const uint64_t one = pair(1.f, 1.f);
      uint64_t wa[4] = {one, one, one, one}, wb[4] = {one, one, one, one};
      if (weight) {
        if (has_a) unpack8<T>(*reinterpret_cast<const uint4*>(weight + 8 * va), wa);
        if (has_b) unpack8<T>(*reinterpret_cast<const uint4*>(weight + 8 * vb), wb);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ka[j] = wa[j];
        kb[j] = wb[j];
        la[j] = lb[j] = 0ull;
        if (INTERLEAVED) {
          // word j of a vector holds one pair: the vector's pairs 4 v + j
          if (turn_a) {
            const float c = j & 1 ? high(cs[j >> 1]) : low(cs[j >> 1]), s = j & 1 ? high(sn[j >> 1]) : low(sn[j >> 1]);
            ka[j] = mul2(wa[j], pair(c, c));
            la[j] = mul2(swap2(wa[j]), pair(-s, s));
          }
          if (turn_b) {
            const float c = j & 1 ? high(cs[2 + (j >> 1)]) : low(cs[2 + (j >> 1)]);
            const float s = j & 1 ? high(sn[2 + (j >> 1)]) : low(sn[2 + (j >> 1)]);
            kb[j] = mul2(wb[j], pair(c, c));
            lb[j] = mul2(swap2(wb[j]), pair(-s, s));
          }
        } else if (turn_a) {
          ka[j] = mul2(wa[j], cs[j]);
          kb[j] = mul2(wb[j], cs[j]);
          la[j] = mul2(wb[j], sn[j] ^ 0x8000000080000000ull);
          lb[j] = mul2(wa[j], sn[j]);
        }
      }
    }
    int h = 4 * (quad - g.first) + (lane >> 3);
    T* to = dst + (long long)h * dst_hs;
    const long long to_step = 4ll * P.parts * dst_hs;
    for (; quad < g.end; quad += P.parts, h += 4 * P.parts, to += to_step) {
      ask();
      cp_async_wait<kAhead - 1>();
      uint4 ua = *reinterpret_cast<const uint4*>(ring + place);
      uint4 ub = *reinterpret_cast<const uint4*>(ring + place + 512);
      place = place + kQuadBytes < kAhead * kQuadBytes ? place + kQuadBytes : 0;
      if (works) {
        uint64_t xa[4], xb[4], ya[4], yb[4];
        if (nv < 16) {                                    // what was never asked for
          if (!has_b) ub = make_uint4(0, 0, 0, 0);
          if (!has_a) ua = make_uint4(0, 0, 0, 0);
        }
        unpack8<T>(ua, xa);
        unpack8<T>(ub, xb);
        uint64_t inv2 = 0ull;
        if (weight) {
          uint64_t ss = mul2(xa[0], xa[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) ss = fma2(xa[j], xa[j], ss);
#pragma unroll
          for (int j = 0; j < 4; ++j) ss = fma2(xb[j], xb[j], ss);
          float sum = low(ss) + high(ss);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
          const float inv = rsqrtf(fmaf(sum, P.inv_dim, P.eps));
          inv2 = pair(inv, inv);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          ya[j] = mul2(xa[j], ka[j]);
          yb[j] = mul2(xb[j], kb[j]);
          if (turn_a) ya[j] = fma2(INTERLEAVED ? swap2(xa[j]) : xb[j], la[j], ya[j]);
          if (turn_b) yb[j] = fma2(INTERLEAVED ? swap2(xb[j]) : xa[j], lb[j], yb[j]);
          if (weight) {
            ya[j] = mul2(ya[j], inv2);
            yb[j] = mul2(yb[j], inv2);
          }
        }
        ua = pack8<T>(ya);
        ub = pack8<T>(yb);
      }
      if (writes && h < g.heads) {
        if (has_a) *reinterpret_cast<uint4*>(to + 8 * va) = ua;
        if (has_b) *reinterpret_cast<uint4*>(to + 8 * vb) = ub;
      }
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
  P.q_quads = (q_heads + 3) / 4;
  P.k_quads = (cache->heads + 3) / 4;
  P.quads = P.q_quads + 2 * P.k_quads;
  // One warp per token when tokens fill the device, so that the angles are
  // computed once for all heads (two warps: 33 us for 25 with 5056 tokens); the
  // quads of a token spread over several warps when they do not (one token: 3.5
  // us for 8.2).
  const long long want = 152ll * 32;
  long long parts = (want + T - 1) / T;
  P.parts = int(parts < 1 ? 1 : parts > P.quads ? P.quads : parts);
  P.by_parts = fast_div(uint32_t(P.parts));
  P.by_page = fast_div(uint32_t(cache->page));
  P.by_share = T % B == 0 ? fast_div(uint32_t(T / B)) : FastDiv{0, 0, 0};
  P.inv_dim = 1.f / float(cache->dim);
  const long long warps = (long long)T * P.parts;
  const unsigned grid = unsigned((warps + kAppThreads / 32 - 1) / (kAppThreads / 32));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = P.interleaved != 0;
  const auto kernel = cache->dtype == DART_F16
                          ? (inter ? append_kernel<__half, true> : append_kernel<__half, false>)
                          : (inter ? append_kernel<__nv_bfloat16, true> : append_kernel<__nv_bfloat16, false>);
  return launch_kernel(kernel, grid, kAppThreads, kRingBytes, s, P) == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
