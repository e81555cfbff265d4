// dart_sample.cu -- K12: tokens drawn from logits with temperature, top-k, top-p and
// min-p, one given random number a row.
//
// Mathematics.  With the row's tokens in descending order of their logits (lower id
// first where they are equal) and w_i = e^((z_i - max) / T), a prefix of that order is
// kept: n = max(1, min(k, n_p, n_m)), n_p the first place where the running sum reaches
// p times the sum of the first k, n_m the number of w_i >= min_p.  The token is the
// first whose running sum exceeds u times the sum of the n kept ones.
//
// Nothing is sorted.  The order is by value, so a histogram of the values answers every
// question of place: a 16-bit logit is its own bin (where its magnitude is usual; the
// rest share three bins), and a bin's weight is its count times the weight of its one
// value.  So a row is read once with an integer add in shared memory for each logit, the
// exponentials are those of a few thousand values, and a second reading (from L2) finds
// the wanted occurrence of the value that was drawn.  Bins of several values (all of
// them where logits have 32 bits) have their weights summed element by element, and the
// one that a place falls into is divided again, 2048 parts at a time, until its parts
// hold one value each.
//
// Which token a random number falls on is a matter of the last bits of sums over the
// whole vocabulary, so weights are 64-bit integers: 2^-y to 2^-45 or better, summed
// exactly in any order.  Results are the same bits every time.
//
// Latency and shared-memory adds bound it, not memory: see the figures at the launch.
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kParts = 2048;                 // of a bin that is divided again

struct SampleParams {
  const void* logits;
  long long stride;
  const float *uniforms, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int R, V, shift;                           // a weight of 1 is 2^shift
};

// Which 16-bit magnitudes have bins of their own: kLow .. kHigh - 1.  bf16: 2^-8 .. 2^9;
// f16: 2^-3 .. 2^6; f32 goes by its upper half, as bf16.
template <typename T> struct Fine { static constexpr int kLow = 119 << 7, kHigh = 136 << 7; };
template <> struct Fine<__half> { static constexpr int kLow = 12 << 10, kHigh = 21 << 10; };

// 2^-j/16 and 2^-j/256 in units of 2^-64.
__constant__ uint64_t kSixteenths[16] = {
    0xffffffffffffffffull, 0xf5257d152486cc2cull, 0xeac0c6e7dd24392full, 0xe0ccdeec2a94e111ull,
    0xd744fccad69d6af4ull, 0xce248c151f8480e4ull, 0xc5672a115506daddull, 0xbd08a39f580c36bfull,
    0xb504f333f9de6484ull, 0xad583eea42a14ac6ull, 0xa5fed6a9b15138eaull, 0x9ef5326091a111aeull,
    0x9837f0518db8a96full, 0x91c3d373ab11c336ull, 0x8b95c1e3ea8bd6e7ull, 0x85aac367cc487b15ull};
__constant__ uint64_t kParts256[16] = {
    0xffffffffffffffffull, 0xff4ecb59511ec8a5ull, 0xfe9e115c7b8f884cull, 0xfdedd1b496a89f35ull,
    0xfd3e0c0cf486c175ull, 0xfc8ec01121e447bbull, 0xfbdfed6ce5f09c49ull, 0xfb3193cc4227c3f4ull,
    0xfa83b2db722a033aull, 0xf9d64a46eb939f35ull, 0xf92959bb5dd4ba74ull, 0xf87ce0e5b2094d9cull,
    0xf7d0df730ad13bb9ull, 0xf7255510c4288239ull, 0xf67a416c733f846eull, 0xf5cfa433e6537290ull};

template <typename T> __device__ __forceinline__ float to_float(uint32_t bits);     // of a 16-bit logit
template <> __device__ __forceinline__ float to_float<__nv_bfloat16>(uint32_t bits) { return __uint_as_float(bits << 16); }
template <> __device__ __forceinline__ float to_float<__half>(uint32_t bits) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
template <> __device__ __forceinline__ float to_float<float>(uint32_t bits) { return __uint_as_float(bits << 16); }

template <typename T>
struct Bins {
  using F = Fine<T>;
  static constexpr int kFine = F::kHigh - F::kLow, kMiddle = kFine + 1, kCount = 2 * kFine + 3;
  static constexpr bool kSingle = sizeof(T) == 2;
  // Bin of a logit by its upper 16 bits, 0 the largest.
  static __device__ __forceinline__ int of(uint32_t bits) {
    const int d = min(max(int(bits & 0x7FFFu), F::kLow - 1), F::kHigh) - (F::kLow - 1);
    return bits & 0x8000u ? kMiddle + d : kMiddle - d;
  }
  static __device__ __forceinline__ bool single(int bin) {
    return kSingle && bin != 0 && bin != kMiddle && bin != kCount - 1;
  }
  // The 16 bits of a bin with a magnitude of its own.
  static __device__ __forceinline__ uint32_t bits(int bin) {
    return bin < kMiddle ? uint32_t(kMiddle - bin + F::kLow - 1) : 0x8000u | uint32_t(bin - kMiddle + F::kLow - 1);
  }
  static __device__ __forceinline__ float value(int bin) { return to_float<T>(bits(bin)); }
  // Ordered keys of the least and largest logit that a bin can hold.
  static __device__ __forceinline__ uint32_t low_key(int bin) {
    if (bin == 0) return ord_f32(to_float<T>(F::kHigh));
    if (bin == kCount - 1) return ord_f32(-3.4028235e38f);
    if (bin == kMiddle) return ~high_key(bin);
    if (kSingle) return ord_f32(value(bin));
    return bin < kMiddle ? ord_f32(value(bin)) : ord_f32(__uint_as_float((bits(bin) << 16) | 0xFFFFu));
  }
  static __device__ __forceinline__ uint32_t high_key(int bin) {
    if (bin == 0) return ord_f32(INFINITY);
    if (bin == kCount - 1) return ord_f32(-to_float<T>(F::kHigh));
    if (bin == kMiddle) return kSingle ? ord_f32(to_float<T>(F::kLow - 1)) : ord_f32(__uint_as_float(((F::kLow - 1) << 16) | 0xFFFFu));
    if (kSingle) return ord_f32(value(bin));
    return bin < kMiddle ? ord_f32(__uint_as_float((bits(bin) << 16) | 0xFFFFu)) : ord_f32(value(bin));
  }
};

// ------------------------------------------------------------------- weights
// e^((z - max) / T) in units of 2^-shift.
struct Weigh {
  float top, c_hi, c_lo;                     // c = log2(e) / T
  int shift;
  const uint64_t* table;                     // 2^-j/256, units of 2^-63
  __device__ __forceinline__ uint64_t operator()(float z) const {
    if (z == top) return 1ull << shift;
    // y = (top - z) c: the difference exactly in two parts, the product in two
    const float d = top - z, v = d - top, e = (top - (d - v)) - (z + v);
    const float y = d * c_hi;
    if (!(y < 62.f)) return 0ull;            // also top = +inf
    const float rest = fmaf(d, c_hi, -y) + fmaf(d, c_lo, e * c_hi);
    // y in units of 2^-48: whole part, 256ths, remainder r
    const long long Y = (long long)(y * 281474976710656.f) + __float2ll_rn(rest * 281474976710656.f);
    if (Y <= 0) return 1ull << shift;
    const int whole = int(Y >> 48), j = int(Y >> 40) & 255;
    // 2^-r = 1 - (x - x^2/2 + x^3/6 - x^4/24), x = r ln 2 < 2^-8, in units of 2^-64; the
    // powers need their upper 32 bits
    const uint64_t x = __umul64hi(uint64_t(Y & ((1ll << 40) - 1)) << 16, 0xb17217f7d1cf79abull);
    const uint32_t a = uint32_t(x >> 24);                              // units of 2^-40
    const uint64_t x2 = (uint64_t(a) * a) >> 17;                       // x^2 / 2
    const uint64_t x3 = (uint64_t(uint32_t(x2 >> 16)) * a) >> 24;      // x^3 / 2
    const uint64_t x4 = (uint64_t(uint32_t(x3 >> 8)) * a) >> 32;       // x^4 / 2
    const uint64_t s = x - x2 + x3 / 3 - x4 / 12;
    const uint64_t t = table[j], w = t - __umul64hi(t, s);
    const int down = 63 - shift + whole;
    return down < 64 ? (w + (1ull << (down - 1))) >> down : 0ull;
  }
};

// ---------------------------------------------------------------- the row
// All threads; f(z) of every logit that counts (not NaN, not -inf), in any order.
template <typename T, typename F>
__device__ __forceinline__ void each_logit(const T* row, int V, F&& f) {
  constexpr int kPer = 16 / int(sizeof(T)), kUnroll = 4;
  const int head = min(V, int((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / int(sizeof(T)));
  const int vecs = (V - head) / kPer, tail = head + vecs * kPer;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  auto one = [&](uint32_t bits, float z) {
    if (z > -INFINITY) f(bits, z);
  };
  auto scalar = [&](int i) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t b = reinterpret_cast<const uint16_t*>(row)[i];
      one(b, to_float<T>(b));
    } else {
      const float z = reinterpret_cast<const float*>(row)[i];
      one(__float_as_uint(z) >> 16, z);
    }
  };
  if (int(threadIdx.x) < head) scalar(threadIdx.x);
  if (tail + int(threadIdx.x) < V) scalar(tail + threadIdx.x);
  for (int v0 = threadIdx.x; v0 < vecs; v0 += kThreads * kUnroll) {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (v0 + u * kThreads < vecs) x[u] = __ldg(body + v0 + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (v0 + u * kThreads >= vecs) break;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 2) {
          one(w[k] & 0xFFFFu, to_float<T>(w[k] & 0xFFFFu));
          one(w[k] >> 16, to_float<T>(w[k] >> 16));
        } else {
          one(w[k] >> 16, __uint_as_float(w[k]));
        }
      }
    }
  }
}

struct Place {                               // of a token in the order
  uint32_t key;                              // its logit
  uint32_t r;                                // tokens of that logit before it
  uint32_t count;                            // tokens of larger logits
  uint64_t weight;                           // their weight
};

struct Shared {
  uint64_t table[256];
  uint64_t warp_weight[kWarps];
  uint32_t warp_count[kWarps];
  uint64_t at_weight;                        // what a search found
  uint32_t at_count, at_bin, at_key, at_r;
  uint32_t part_count[kParts];
  uint64_t part_weight[kParts];
};

// Exclusive sums over the CTA's threads, and the totals.
__device__ __forceinline__ void scan(Shared* sh, uint32_t& c, uint64_t& w, uint32_t& total_c, uint64_t& total_w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t ci = c;
  uint64_t wi = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t cx = __shfl_up_sync(kFull, ci, o);
    const uint64_t wx = __shfl_up_sync(kFull, wi, o);
    if (lane >= o) {
      ci += cx;
      wi += wx;
    }
  }
  __syncthreads();
  if (lane == 31) {
    sh->warp_count[warp] = ci;
    sh->warp_weight[warp] = wi;
  }
  __syncthreads();
  uint32_t cb = 0;
  uint64_t wb = 0;
  total_c = 0;
  total_w = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) {
      cb = total_c;
      wb = total_w;
    }
    total_c += sh->warp_count[i];
    total_w += sh->warp_weight[i];
  }
  c = cb + ci - c;
  w = wb + wi - w;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams P) {
  using B = Bins<T>;
  constexpr int kPer = (B::kCount + kThreads - 1) / kThreads;       // bins of a thread
  static_assert(kPer <= 64, "a warp looks at a thread's bins in two steps");
  extern __shared__ __align__(16) unsigned char smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem);
  uint64_t* bin_weight = reinterpret_cast<uint64_t*>(sh + 1);       // of bins of several values: all, or three
  uint32_t* bin_count = reinterpret_cast<uint32_t*>(bin_weight + (B::kSingle ? 4 : B::kCount + 1));
  auto slot = [](int bin) { return B::kSingle ? (bin == 0 ? 0 : bin == B::kMiddle ? 1 : 2) : bin; };

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / P.R, V = P.V;
  const T* row = static_cast<const T*>(P.logits) + (long long)blockIdx.x * P.stride;
  const float heat = P.temperature ? P.temperature[b] : 1.f;
  const int top_k = P.top_k ? P.top_k[b] : 0;
  const float top_p = P.top_p ? P.top_p[b] : 1.f, min_p = P.min_p ? P.min_p[b] : 0.f;
  const bool greedy = !(heat > 0.f) || top_k == 1 || top_p <= 0.f || min_p > 1.f;

  // ---- counts of all bins, and the largest logit
  if (!greedy) {
    for (int i = tid; i < B::kCount; i += kThreads) bin_count[i] = 0;
    for (int i = tid; i < (B::kSingle ? 4 : B::kCount); i += kThreads) bin_weight[i] = 0;
    if (tid < 256) sh->table[tid] = __umul64hi(kSixteenths[tid >> 4], kParts256[tid & 15]) >> 1;
    __syncthreads();
  }
  float top = -INFINITY;
  if (greedy)
    each_logit(row, V, [&](uint32_t, float z) { top = fmaxf(top, z); });
  else
    each_logit(row, V, [&](uint32_t bits, float z) {
      top = fmaxf(top, z);
      atomicAdd(&bin_count[B::of(bits)], 1u);
    });
  {
    const uint32_t key = __reduce_max_sync(kFull, ord_f32(top));
    if (lane == 0) sh->warp_count[warp] = key;
    __syncthreads();
    uint32_t best = sh->warp_count[lane % kWarps];
    best = __reduce_max_sync(kFull, best);
    top = unord_f32(best);
    __syncthreads();
  }
  if (top == -INFINITY) {                    // nothing is left to draw from
    if (tid == 0) {
      P.tokens[blockIdx.x] = -1;
      P.probs[blockIdx.x] = 0.f;
    }
    return;
  }

  Place drawn{ord_f32(top), 0u, 0u, 0ull};
  float prob = 1.f;
  if (!greedy) {
    Weigh weigh;
    weigh.top = top;
    weigh.shift = P.shift;
    weigh.table = sh->table;
    // beyond 2^100 every logit but the largest weighs nothing anyway
    const double c = fmin(1.4426950408889634 / double(heat), 1.2676506002282294e30);
    weigh.c_hi = float(c);
    weigh.c_lo = float(c - double(weigh.c_hi));

    // ---- places by count
    const int bin0 = min(tid * kPer, B::kCount), bin1 = min(bin0 + kPer, B::kCount);
    uint32_t count0 = 0, total;
    uint64_t weight0 = 0, all;
    for (int i = bin0; i < bin1; ++i) count0 += bin_count[i];
    const uint32_t mine = count0;
    scan(sh, count0, weight0, total, all);
    uint32_t enough = total;                 // n_m
    if (min_p > 0.f) {
      // w >= min_p where z >= max + T ln(min_p)
      const float least = __double2float_ru(double(top) + double(heat) * log(double(min_p)));
      const uint32_t key = ord_f32(least);
      uint32_t n = 0;
      bool cut = false;
      for (int i = bin0; i < bin1; ++i) {
        if (bin_count[i] == 0) continue;
        if (B::low_key(i) >= key) n += bin_count[i];
        else if (B::high_key(i) >= key) cut = true;
      }
      uint32_t zero = 0;
      uint64_t none = 0;
      scan(sh, n, none, enough, all);
      if (__syncthreads_or(cut)) {
        // the bin that the limit falls into, element by element
        each_logit(row, V, [&](uint32_t bits, float z) {
          if (z >= least && B::low_key(B::of(bits)) < key) ++zero;
        });
        uint32_t more;
        none = 0;
        scan(sh, zero, none, more, all);
        enough += more;
      }
      enough = max(enough, 1u);
    }
    const uint32_t most = top_k > 0 ? min(uint32_t(top_k), total) : total;
    const bool by_p = top_p < 1.f;
    const uint32_t last = by_p ? most : min(most, enough);          // weights are wanted up to this place
    if (count0 < last && last <= count0 + mine) {
      uint32_t n = count0;
      int i = bin0;
      while (n + bin_count[i] < last) n += bin_count[i++];
      sh->at_bin = uint32_t(i);
    }
    __syncthreads();
    const int last_bin = int(sh->at_bin);

    // ---- weights of the bins up to there
    bool several = false;
    for (int i = bin0; i < min(bin1, last_bin + 1); ++i) several |= !B::single(i) && bin_count[i] > 0;
    if (__syncthreads_or(several))
      each_logit(row, V, [&](uint32_t bits, float z) {
        const int i = B::of(bits);
        if (i <= last_bin && !B::single(i))
          atomicAdd(reinterpret_cast<unsigned long long*>(&bin_weight[slot(i)]), (unsigned long long)weigh(z));
      });
    __syncthreads();
    auto weight_of = [&](int i) -> uint64_t {
      const uint32_t n = bin_count[i];
      if (n == 0) return 0ull;
      return B::single(i) ? n * weigh(B::value(i)) : bin_weight[slot(i)];
    };
    weight0 = 0;
    for (int i = bin0; i < min(bin1, last_bin + 1); ++i) weight0 += weight_of(i);
    uint64_t own = weight0;
    {
      uint32_t c = 0, cc;
      scan(sh, c, weight0, cc, all);
    }

    // The place of the token before which there are x tokens (by_count), or the first
    // whose running sum exceeds x.  All threads.
    auto find = [&](bool by_count, uint64_t x) -> Place {
      const bool here = by_count ? count0 <= x && x < uint64_t(count0) + mine : weight0 <= x && x < weight0 + own;
      __syncthreads();
      if (here) {
        sh->at_bin = uint32_t(bin0);
        sh->at_count = count0;
        sh->at_weight = weight0;
      }
      __syncthreads();
      Place at;
      int bin = int(sh->at_bin);
      at.count = sh->at_count;
      at.weight = sh->at_weight;
      // every warp looks at that thread's bins
      const int end = min(bin + kPer, B::kCount);
      for (int i0 = bin; i0 < end; i0 += 32) {
        const int i = i0 + lane;
        uint32_t c = i < end ? bin_count[i] : 0u;
        uint64_t w = i < end && i <= last_bin ? weight_of(i) : 0ull;
        const uint32_t c1 = c;
        const uint64_t w1 = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t cx = __shfl_up_sync(kFull, c, o);
          const uint64_t wx = __shfl_up_sync(kFull, w, o);
          if (lane >= o) {
            c += cx;
            w += wx;
          }
        }
        const uint32_t hit = __ballot_sync(kFull, by_count ? x < uint64_t(at.count) + c : x < at.weight + w);
        const int l = hit ? __ffs(hit) - 1 : 31;
        bin = i0 + l;
        const uint32_t add_c = __shfl_sync(kFull, hit ? c - c1 : c, l);
        const uint64_t add_w = __shfl_sync(kFull, hit ? w - w1 : w, l);
        at.count += add_c;
        at.weight += add_w;
        if (hit) break;
      }
      at.key = B::high_key(bin);
      if (!B::single(bin)) {
        // divided again until a part is one value
        uint32_t lo = B::low_key(bin), hi = at.key;
        for (;;) {
          const uint32_t span = hi - lo;
          const int bits = span ? 32 - __clz(span) : 0, down = bits > 11 ? bits - 11 : 0;
          __syncthreads();
          for (int i = tid; i < kParts; i += kThreads) {
            sh->part_count[i] = 0;
            sh->part_weight[i] = 0;
          }
          __syncthreads();
          each_logit(row, V, [&](uint32_t, float z) {
            const uint32_t key = ord_f32(z);
            if (key >= lo && key <= hi) {
              const uint32_t i = (hi - key) >> down;
              atomicAdd(&sh->part_count[i], 1u);
              atomicAdd(reinterpret_cast<unsigned long long*>(&sh->part_weight[i]), (unsigned long long)weigh(z));
            }
          });
          __syncthreads();
          constexpr int kEach = kParts / kThreads;
          uint32_t c = 0, cc;
          uint64_t w = 0, ww;
          for (int k = 0; k < kEach; ++k) {
            c += sh->part_count[tid * kEach + k];
            w += sh->part_weight[tid * kEach + k];
          }
          scan(sh, c, w, cc, ww);
          c += at.count;
          w += at.weight;
          for (int k = 0; k < kEach; ++k) {
            const uint32_t n = sh->part_count[tid * kEach + k];
            const uint64_t m = sh->part_weight[tid * kEach + k];
            if (by_count ? c <= x && x < uint64_t(c) + n : w <= x && x < w + m) {
              sh->at_bin = uint32_t(tid * kEach + k);
              sh->at_count = c;
              sh->at_weight = w;
            }
            c += n;
            w += m;
          }
          __syncthreads();
          hi -= sh->at_bin << down;
          lo = max(lo, hi - ((1u << down) - 1u));
          at.count = sh->at_count;
          at.weight = sh->at_weight;
          if (down == 0) break;
        }
        at.key = hi;
      }
      at.r = by_count ? uint32_t(x - at.count) : uint32_t((x - at.weight) / weigh(unord_f32(at.key)));
      return at;
    };
    // the weight up to and with the token at a place
    auto upto = [&](const Place& at) { return at.weight + (uint64_t(at.r) + 1) * weigh(unord_f32(at.key)); };

    uint64_t sum = all;                      // of the first `most`
    if (most < total && (by_p || most <= enough)) sum = upto(find(true, most - 1));
    uint32_t n = most;
    if (by_p) {
      // the first place where the running sum is at least p times the sum
      uint64_t reach = uint64_t(ceil(double(top_p) * double(sum)));
      reach = reach < 1 ? 1 : reach > sum ? sum : reach;
      const Place at = find(false, reach - 1);
      n = at.count + at.r + 1;
      sum = upto(at);
    }
    if (enough < n) {
      n = enough;
      sum = upto(find(true, n - 1));
    }
    const float u = P.uniforms[blockIdx.x];
    uint64_t x = u > 0.f ? uint64_t(double(u) * double(sum)) : 0ull;
    if (x >= sum) x = sum - 1;
    drawn = find(false, x);
    prob = float(double(weigh(unord_f32(drawn.key))) / double(sum));
  }

  // ---- the drawn.r-th token (from 0) of that logit in the order of ids
  const float z = unord_f32(drawn.key);
  constexpr int kVec = 16 / int(sizeof(T));
  const int head = min(V, int((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / int(sizeof(T)));
  const int vecs = (V - head) / kVec, tail = head + vecs * kVec;
  const uint4* body = reinterpret_cast<const uint4*>(row + head);
  auto matches = [&](const uint4& x) -> uint32_t {           // a bit for each element of a vector
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 2) {
        m |= (to_float<T>(w[k] & 0xFFFFu) == z ? 1u : 0u) << (2 * k);
        m |= (to_float<T>(w[k] >> 16) == z ? 1u : 0u) << (2 * k + 1);
      } else {
        m |= (__uint_as_float(w[k]) == z ? 1u : 0u) << k;
      }
    }
    return m;
  };
  // warp w has the vectors from w share to (w + 1) share; the head is before them, the tail behind
  const int share = (vecs + kWarps - 1) / kWarps, v0 = min(warp * share, vecs), v1 = min(v0 + share, vecs);
  uint32_t n = 0;
  for (int v = v0 + lane; v < v1; v += 32 * 4) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + 32 * k < v1) x[k] = __ldg(body + v + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + 32 * k < v1) n += __popc(matches(x[k]));
  }
  n = __reduce_add_sync(kFull, n);
  __syncthreads();
  if (lane == 0) sh->warp_count[warp] = n;
  __syncthreads();
  if (warp != 0) return;
  uint32_t left = drawn.r;
  int token = -1;
  auto singly = [&](int i0, int i1) {
    for (int i = i0; i < i1 && token < 0; ++i)
      if (float(row[i]) == z) {
        if (left == 0) token = i;
        else --left;
      }
  };
  singly(0, head);
  if (token < 0) {
    int w = 0;
    while (w < kWarps && left >= sh->warp_count[w]) left -= sh->warp_count[w++];
    if (w < kWarps) {
      const int first = min(w * share, vecs), end = min(first + share, vecs);
      for (int v = first; v < end; v += 32) {
        const uint32_t m = v + lane < end ? matches(__ldg(body + v + lane)) : 0u;
        uint32_t c = __popc(m);
        const uint32_t c1 = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(kFull, c, o);
          if (lane >= o) c += y;
        }
        const uint32_t in_step = __shfl_sync(kFull, c, 31);
        if (left < in_step) {
          int at = -1;
          if (left >= c - c1 && left < c) {
            uint32_t bits = m;
            for (uint32_t k = left - (c - c1); k > 0; --k) bits &= bits - 1;
            at = head + (v + lane) * kVec + __ffs(bits) - 1;
          }
          token = __reduce_max_sync(kFull, at);
          break;
        }
        left -= in_step;
      }
    } else {
      singly(tail, V);
    }
  }
  if (lane == 0) {
    P.tokens[blockIdx.x] = token;
    P.probs[blockIdx.x] = prob;
  }
}

template <typename T>
cudaError_t launch(const SampleParams& P, long long rows, cudaStream_t s) {
  using B = Bins<T>;
  const int smem = int(sizeof(Shared)) + 8 * (B::kSingle ? 4 : B::kCount + 1) + 4 * B::kCount;
  const cudaError_t e = settled(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (e != cudaSuccess) return e;
  return launch_kernel(sample_kernel<T>, unsigned(rows), kThreads, smem, s, P);
}

}  // namespace
}  // namespace dart

extern "C" int dart_logits_sample(const void* logits, int B, int R, int V, int64_t row_stride, int dtype,
                                  const float* uniforms, const float* temperature, const int32_t* top_k,
                                  const float* top_p, const float* min_p, int32_t* out_tokens, float* out_probs,
                                  void* stream) {
  using namespace dart;
  if (B < 0 || R < 0 || V < 1 || V > kMaxV || row_stride < V || row_stride > kMaxRowStride) return DART_ERR_INVALID_ARG;
  if (dtype != DART_F32 && dtype != DART_F16 && dtype != DART_BF16) return DART_ERR_INVALID_ARG;
  const long long rows = (long long)B * R;
  if (rows >= (1ll << 31)) return DART_ERR_INVALID_ARG;
  if (rows == 0) return DART_OK;
  const int size = dtype == DART_F32 ? 4 : 2;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size != 0 || !uniforms || !out_tokens || !out_probs)
    return DART_ERR_INVALID_ARG;
  int bits = 1;
  while ((1ll << bits) <= V) ++bits;
  SampleParams P;
  P.logits = logits; P.stride = row_stride;
  P.uniforms = uniforms; P.temperature = temperature; P.top_p = top_p; P.min_p = min_p; P.top_k = top_k;
  P.tokens = out_tokens; P.probs = out_probs;
  P.R = R; P.V = V;
  P.shift = 62 - bits;                       // the sum of V weights of 1 stays below 2^62
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DART_F32   ? launch<float>(P, rows, s)
                        : dtype == DART_F16 ? launch<__half>(P, rows, s)
                                            : launch<__nv_bfloat16>(P, rows, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
