// dart_adjust.cu -- K5: penalties for repeated tokens, biases and grammar
// masks on logits, in one pass from the input rows to the output rows.
//
// What a row needs beyond its own elements is small and shared: how often each
// token occurs in the sequence's history, and the summed bias of each token.
// So a CTA owns a slice of the vocabulary of one sequence, counts the history
// and sums the biases of that slice in shared memory once, and then streams
// that slice of its rows.  A bitmap of the tokens that are counted or biased
// lets every other element pass unexamined, and a vector of elements that the
// grammar bans is written without being read.
#include <atomic>
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjVecs = 4;                                // 16-byte vectors a lane takes of a row
constexpr int kMaxBias = 1024;                             // biases per sequence
constexpr unsigned kFull = 0xFFFFFFFFu;

// A vector per lane makes a block of tokens (256 of 16 bits, 128 of 32).  The
// blocks of the vocabulary are dealt to the CTAs in turn and a CTA's blocks to
// its warps in turn, because the tokens that are counted crowd together at low
// ids and a block that holds any takes several times as long.
template <typename T> constexpr int kBlock = 32 * (16 / int(sizeof(T)));
template <typename T> constexpr int kSlice = kAdjWarps * kAdjVecs * kBlock<T>;

struct AdjustParams {
  const void* in;
  void* out;
  int R, V, row_group;                 // rows per CTA
  long long in_stride, out_stride;
  dart_adjust_t a;
  bool count;                          // some penalty is given
  FastDiv by_slices;                   // slices of the vocabulary: block k belongs to slice k % slices
};

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
  static constexpr uint32_t kNegInf = 0xFF800000u;
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
  static constexpr uint32_t kNegInf = 0xFC00FC00u;
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
};

template <typename T>
union Vec {
  uint4 u;
  T e[16 / sizeof(T)];
};

// Logits pass through once: keep them out of the way of what is used again.
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void stg_stream(void* p, uint4 v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};"
               :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 32 bits from bit `at` on of an array of `words` words (those behind it are 0).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int at, int words) {
  const int i = at >> 5;
  const uint32_t lo = w[i];
  if ((at & 31) == 0) return lo;
  const uint32_t hi = i + 1 < words ? w[i + 1] : 0u;
  return __funnelshift_r(lo, hi, at & 31);
}

// The vector with -inf in the places whose bit of `keep` is clear.
template <typename T>
__device__ __forceinline__ uint4 ban(uint4 u, uint32_t keep) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t m;
    if (sizeof(T) == 2) {
      const uint32_t t = keep >> (2 * j);
      const uint32_t u2 = (t | (t << 15)) & 0x00010001u;      // the two bits, one in each half
      m = (u2 << 16) - u2;                                    // 0xFFFF in each kept half
    } else {
      m = 0u - ((keep >> j) & 1u);
    }
    w[j] = (w[j] & m) | (Elem<T>::kNegInf & ~m);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// ALIGNED: every row begins on a 16-byte boundary, in and out.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kAdjThreads, 3)
adjust_kernel(const AdjustParams P) {
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kBlk = kBlock<T>, kCta = kSlice<T>, kWords = kCta / 32;
  constexpr uint32_t kAll = (1u << E) - 1u;
  extern __shared__ __align__(16) unsigned char smem[];
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem);                    // [kCta], with penalties
  float* bias = reinterpret_cast<float*>(smem) + (P.count ? kCta : 0);     // [kCta], with biases
  __shared__ __align__(16) uint32_t touched[kWords + 1];         // token is counted or biased
  __shared__ uint32_t bias_bits[kWords + 1];       // token is biased
  __shared__ int32_t list_id[kMaxBias];            // the slice's biases, in their order; then the tree's tokens
  __shared__ float list_val[kMaxBias];
  __shared__ int32_t warp_n[kMaxBias / kAdjThreads][kAdjWarps];
  static_assert(kMaxN <= kMaxBias, "the tree's tokens take the place of the bias list");

  const int b = blockIdx.z, slice = blockIdx.x, slices = int(P.by_slices.d);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const dart_adjust_t& a = P.a;
  // token -> its place in the slice, -1 if it belongs to another or to none
  auto local = [&](int32_t token) {
    const int blk = token / kBlk, k = P.by_slices.div(blk);
    return uint32_t(token) < uint32_t(P.V) && blk - k * slices == slice ? k * kBlk + token % kBlk : -1;
  };

  // Everything that the slice needs from memory is asked for before anything waits.
  constexpr int kAhead = 8, kBiasAhead = kMaxBias / kAdjThreads;
  const int32_t* hist = P.count && a.history ? a.history + (long long)b * a.history_stride : nullptr;
  const int width = hist ? a.history_width : 0;
  int32_t id[kAhead], bias_id[kBiasAhead];
  float bias_val[kBiasAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) id[k] = tid + k * kAdjThreads < width ? hist[tid + k * kAdjThreads] : -1;
#pragma unroll
  for (int k = 0; k < kBiasAhead; ++k) {
    const int i = tid + k * kAdjThreads;
    bias_id[k] = i < a.bias_count ? a.bias_ids[(long long)b * a.bias_count + i] : -1;
    bias_val[k] = i < a.bias_count ? a.bias_vals[(long long)b * a.bias_count + i] : 0.f;
  }
  const int len = hist ? (a.history_len ? max(0, min(a.history_len[b], width)) : width) : 0;
  const float rep = a.repetition ? a.repetition[b] : 1.f, inv_rep = 1.f / rep;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;

  for (int i = tid; i <= kWords; i += kAdjThreads) touched[i] = bias_bits[i] = 0u;
  {
    uint4* z = reinterpret_cast<uint4*>(smem);
    const int n = ((P.count ? 1 : 0) + (a.bias_count > 0 ? 1 : 0)) * (kCta / 4);
    for (int i = tid; i < n; i += kAdjThreads) z[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  for (int i0 = tid; i0 < len; i0 += kAhead * kAdjThreads) {
    if (i0 != tid) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) id[k] = i0 + k * kAdjThreads < len ? hist[i0 + k * kAdjThreads] : -1;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int t = i0 + k * kAdjThreads < len ? local(id[k]) : -1;
      if (t >= 0) {
        atomicAdd(&counts[t], 1u);
        atomicOr(&touched[t >> 5], 1u << (t & 31));
      }
    }
  }
  if (a.bias_count > 0) {
    // The slice's biases, compacted in their order; then the first entry of
    // each id sums that id's values in order, so that repeated ids always give
    // the same sum.
    int n = 0;
#pragma unroll
    for (int k = 0; k < kBiasAhead; ++k) {
      if (k * kAdjThreads >= a.bias_count) break;
      const int t = local(bias_id[k]);
      const unsigned m = __ballot_sync(kFull, t >= 0);
      if (lane == 0) warp_n[k][warp] = __popc(m);
      __syncthreads();
      int at = n + __popc(m & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kAdjWarps; ++w) {
        if (w < warp) at += warp_n[k][w];
        n += warp_n[k][w];
      }
      if (t >= 0) {
        list_id[at] = t;
        list_val[at] = bias_val[k];
      }
    }
    __syncthreads();
    for (int i = tid; i < n; i += kAdjThreads) {
      const int32_t t = list_id[i];
      bool first = true;
      for (int j = 0; j < i; ++j) first &= list_id[j] != t;
      if (!first) continue;
      float s = list_val[i];
      for (int j = i + 1; j < n; ++j)
        if (list_id[j] == t) s += list_val[j];
      bias[t] = s;
      atomicOr(&bias_bits[t >> 5], 1u << (t & 31));
      atomicOr(&touched[t >> 5], 1u << (t & 31));
    }
  }
  const int r_begin = blockIdx.y * P.row_group, r_end = min(P.R, r_begin + P.row_group);
  const bool paths = P.count && a.N > 0;
  int32_t* toks = list_id;                       // from here on: the places of the tree's tokens in the slice
  if (paths) {
    __syncthreads();
    for (int i = tid; i < a.N; i += kAdjThreads) toks[i] = local(a.tokens[(long long)b * a.N + i]);
  }
  __syncthreads();

  // From here on a warp touches its own blocks only: block i lies at place
  // (8 i + warp) * kBlk of the slice and holds the tokens from token(i) on.
  auto place = [&](int i) { return (kAdjWarps * i + warp) * kBlk; };
  auto token = [&](int i) { return ((kAdjWarps * i + warp) * slices + slice) * kBlk; };
  auto size = [&](int i) { return min(P.V - token(i), kBlk); };          // <= 0 behind the vocabulary
  if (token(0) >= P.V) return;
  const int words = (P.V + 31) >> 5;
  const int MW = (a.N + 31) >> 5;
  const bool biased = a.bias_count > 0;

  // the nodes whose tokens this warp owns, 32 nodes a lane
  uint32_t own_nodes = 0u;
  auto owns = [&](int node) { return toks[node] >= 0 && toks[node] / kBlk % kAdjWarps == warp; };
  if (paths)
    for (int k = 0; k < 32 && 32 * lane + k < a.N; ++k) own_nodes |= uint32_t(owns(32 * lane + k)) << k;
  auto node_bits = [&](int r) {       // this lane's word of the row's path
    const int node = r - (P.R - a.N);
    return paths && r < r_end && node >= 0 && lane < MW ? a.mask[((long long)b * a.N + node) * MW + lane] : 0u;
  };
  // the tokens of the row's path join the counts, and leave them again
  auto path_in = [&](uint32_t m) {
    for (; m; m &= m - 1) {
      const int t = toks[32 * lane + __ffs(m) - 1];
      atomicAdd(&counts[t], 1u);
      atomicOr(&touched[t >> 5], 1u << (t & 31));
    }
    __syncwarp();
  };
  auto path_out = [&](uint32_t m) {
    __syncwarp();
    for (; m; m &= m - 1) {
      const int t = toks[32 * lane + __ffs(m) - 1];
      if (atomicSub(&counts[t], 1u) == 1u && !((bias_bits[t >> 5] >> (t & 31)) & 1u))
        atomicAnd(&touched[t >> 5], ~(1u << (t & 31)));
    }
    __syncwarp();
  };

  // element x with count c and bias y (0: not biased, as far as the value goes)
  auto apply = [&](float x, uint32_t c, float y) {
    const float z = fmaf(-freq, float(c), x > 0.f ? x * inv_rep : x * rep) - pres;
    return (c ? z : x) + y;
  };
  // one element: token v, at place t of the slice
  auto scalar = [&](const T* in, T* out, const uint32_t* allow, int v, int t) {
    const uint32_t word = allow ? allow[v >> 5] : kFull;
    T x;
    if ((word >> (v & 31)) & 1u) {
      x = in[v];
      if ((touched[t >> 5] >> (t & 31)) & 1u)
        x = Elem<T>::put(apply(Elem<T>::get(x), P.count ? counts[t] : 0u, biased ? bias[t] : 0.f));
    } else {
      x = Elem<T>::put(-INFINITY);
    }
    out[v] = x;
  };
  // the elements `hit` of the vector at place t (a multiple of 4 if ALIGNED)
  auto adjust_vec = [&](Vec<T>& x, uint32_t hit, int t) {
    uint32_t c[E];
    float y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = 0u, y[e] = 0.f;
    if constexpr (ALIGNED) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        if (P.count) *reinterpret_cast<uint4*>(c + e) = *reinterpret_cast<const uint4*>(counts + t + e);
        if (biased) *reinterpret_cast<float4*>(y + e) = *reinterpret_cast<const float4*>(bias + t + e);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (P.count) c[e] = counts[t + e];
        if (biased) y[e] = bias[t + e];
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((hit >> e) & 1u) x.e[e] = Elem<T>::put(apply(Elem<T>::get(x.e[e]), c[e], y[e]));
  };

  const T* in = static_cast<const T*>(P.in) + ((long long)b * P.R + r_begin) * P.in_stride;
  T* out = static_cast<T*>(P.out) + ((long long)b * P.R + r_begin) * P.out_stride;
  const uint32_t* allow =
      a.allowed ? a.allowed + (long long)b * a.allowed_seq_stride + (long long)r_begin * a.allowed_row_stride : nullptr;
  uint32_t path = node_bits(r_begin);

  if constexpr (ALIGNED) {
    // The lane's vectors lie `step` tokens apart, from v0 on; the first `nv` of
    // them are whole.  The next row's grammar bits come while this one is worked on.
    const int step = kAdjWarps * slices * kBlk, v0 = token(0) + lane * E, t0 = place(0) + lane * E;
    int nv = 0;
#pragma unroll
    for (int i = 0; i < kAdjVecs; ++i) nv += v0 + i * step + E <= P.V ? 1 : 0;
    // tokens behind the last whole vector of the vocabulary, the warp that owns them taking them singly
    const int rest = P.V % E, rest0 = P.V - rest, rest_at = local(rest0);
    const bool mine = rest > 0 && lane < rest && rest_at >= 0 && rest_at / kBlk % kAdjWarps == warp;
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(touched) + (t0 >> 3);
    const int shift = t0 & 7;                     // a vector of four shares its byte with its neighbour
    auto grammar = [&](const uint32_t* al) {      // eight bits per vector
      uint32_t ok = 0u;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(al) + (v0 >> 3);
#pragma unroll
      for (int i = 0; i < kAdjVecs; ++i)
        if (i < nv) ok |= ((uint32_t(src[i * (step / 8)]) >> shift) & kAll) << (8 * i);
      return ok;
    };
    uint32_t ok = allow ? grammar(allow) : kFull;
    in += v0;
    out += v0;
    for (int r = r_begin; r < r_end; ++r) {
      Vec<T> x[kAdjVecs];
#pragma unroll
      for (int i = 0; i < kAdjVecs; ++i)
        if (i < nv && ((ok >> (8 * i)) & kAll)) x[i].u = ldg_stream(in + i * step);
      const uint32_t next_path = node_bits(r + 1);
      uint32_t next_ok = kFull;
      if (allow && r + 1 < r_end) next_ok = grammar(allow + a.allowed_row_stride);
      const uint32_t m = path & own_nodes;
      const bool walked = paths && __any_sync(kFull, m != 0u);
      if (walked) path_in(m);
#pragma unroll
      for (int i = 0; i < kAdjVecs; ++i) {
        if (i < nv) {
          const uint32_t keep = (ok >> (8 * i)) & kAll;
          const uint32_t hit = (uint32_t(bytes[i * (kAdjWarps * kBlk / 8)]) >> shift) & keep;
          if (hit) adjust_vec(x[i], hit, t0 + i * (kAdjWarps * kBlk));
          if (allow) x[i].u = ban<T>(x[i].u, keep);
          stg_stream(out + i * step, x[i].u);
        }
      }
      if (mine) scalar(in - v0, out - v0, allow, rest0 + lane, rest_at + lane);
      if (walked) path_out(m);
      in += P.in_stride;
      out += P.out_stride;
      if (allow) allow += a.allowed_row_stride;
      ok = next_ok;
      path = next_path;
    }
  } else {
    for (int r = r_begin; r < r_end; ++r) {
      const uint32_t m = path & own_nodes;
      path = node_bits(r + 1);
      const bool walked = paths && __any_sync(kFull, m != 0u);
      if (walked) path_in(m);
      // elements before the first 16-byte boundary of every block of this row (a block is a multiple of 16 bytes)
      const int head = int((16u - unsigned(reinterpret_cast<uintptr_t>(in) & 15u)) & 15u) / int(sizeof(T));
      const bool same = ((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
      if (same) {
        uint32_t ok[kAdjVecs];
        Vec<T> x[kAdjVecs];
#pragma unroll
        for (int i = 0; i < kAdjVecs; ++i) {
          const int v = token(i) + head + lane * E;
          ok[i] = head + (lane + 1) * E <= size(i) ? (allow ? bits_at(allow, v, words) & kAll : kAll) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kAdjVecs; ++i)
          if (ok[i]) x[i].u = ldg_stream(in + token(i) + head + lane * E);
#pragma unroll
        for (int i = 0; i < kAdjVecs; ++i) {
          const int n = size(i), t = place(i) + head + lane * E;
          if (head + (lane + 1) * E <= n) {
            const uint32_t hit = bits_at(touched, t, kWords + 1) & ok[i];
            if (hit) adjust_vec(x[i], hit, t);
            if (allow) x[i].u = ban<T>(x[i].u, ok[i]);
            stg_stream(out + token(i) + head + lane * E, x[i].u);
          }
          if (lane < min(head, n)) scalar(in, out, allow, token(i) + lane, place(i) + lane);
          const int tail = head < n ? head + (n - head) / E * E : max(n, 0);
          if (lane < n - tail) scalar(in, out, allow, token(i) + tail + lane, place(i) + tail + lane);
        }
      } else {
        for (int i = 0; i < kAdjVecs; ++i)
          for (int k = lane; k < size(i); k += 32) scalar(in, out, allow, token(i) + k, place(i) + k);
      }
      if (walked) path_out(m);
      in += P.in_stride;
      out += P.out_stride;
      if (allow) allow += a.allowed_row_stride;
    }
  }
}

template <typename T, bool ALIGNED>
cudaError_t raise_limit() {
  static std::atomic<uint64_t> ready{0};       // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!bit || !(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(adjust_kernel<T, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kSlice<T>);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  }
  return e;
}

template <typename T>
cudaError_t launch_adjust(AdjustParams P, int B, cudaStream_t stream) {
  const uintptr_t low = reinterpret_cast<uintptr_t>(P.in) | reinterpret_cast<uintptr_t>(P.out) |
                        uintptr_t((P.in_stride | P.out_stride) * int(sizeof(T)));
  const bool aligned = (low & 15) == 0;
  const cudaError_t e = aligned ? raise_limit<T, true>() : raise_limit<T, false>();
  if (e != cudaSuccess) return e;
  const int slices = (P.V + kSlice<T> - 1) / kSlice<T>;
  P.by_slices = fast_div(uint32_t(slices));
  // rows per CTA: enough CTAs to fill the device a few times, then as many rows
  // as possible share one count
  const long long want = 152ll * 3 * 2, per = (long long)slices * B;
  long long groups = (want + per - 1) / per;
  groups = groups > P.R ? P.R : groups;
  if (groups > 65535) groups = 65535;
  P.row_group = int((P.R + groups - 1) / groups);
  const dim3 grid(slices, (P.R + P.row_group - 1) / P.row_group, B);
  const size_t smem = size_t(4 * kSlice<T>) * ((P.count ? 1 : 0) + (P.a.bias_count > 0 ? 1 : 0));
  if (aligned) adjust_kernel<T, true><<<grid, kAdjThreads, smem, stream>>>(P);
  else adjust_kernel<T, false><<<grid, kAdjThreads, smem, stream>>>(P);
  return cudaGetLastError();
}

}  // namespace
}  // namespace dart

extern "C" int dart_logits_adjust(const void* logits, int B, int R, int V, int64_t row_stride, int dtype,
                                  const dart_adjust_t* what, void* out, int64_t out_stride, void* stream) {
  using namespace dart;
  if (!what || what->reserved != 0 || B < 0 || B > 65535 || R < 0 || V < 1 || V > kMaxV) return DART_ERR_INVALID_ARG;
  if (dtype != DART_F32 && dtype != DART_F16 && dtype != DART_BF16) return DART_ERR_INVALID_ARG;
  if (row_stride < V || row_stride > kMaxRowStride || out_stride < V || out_stride > kMaxRowStride)
    return DART_ERR_INVALID_ARG;
  const dart_adjust_t& a = *what;
  if (a.history_width < 0 || a.bias_count < 0 || a.bias_count > kMaxBias || a.N < 0 || a.N > kMaxN)
    return DART_ERR_INVALID_ARG;
  if (a.history && a.history_stride < a.history_width && B > 1) return DART_ERR_INVALID_ARG;
  if (a.N > 0 && R != a.N && R != a.N + 1) return DART_ERR_INVALID_ARG;
  if (a.allowed && (a.allowed_seq_stride < 0 || a.allowed_row_stride < 0)) return DART_ERR_INVALID_ARG;
  if (B == 0 || R == 0) return DART_OK;
  if (a.bias_count > 0 && (!a.bias_ids || !a.bias_vals)) return DART_ERR_INVALID_ARG;
  if (a.N > 0 && (!a.tokens || !a.mask)) return DART_ERR_INVALID_ARG;
  const uintptr_t es = dtype == DART_F32 ? 4 : 2;
  if (!logits || !out || reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % es)
    return DART_ERR_INVALID_ARG;
  if (logits == out && row_stride != out_stride) return DART_ERR_INVALID_ARG;
  AdjustParams P;
  P.in = logits;
  P.out = out;
  P.R = R;
  P.V = V;
  P.in_stride = row_stride;
  P.out_stride = out_stride;
  P.a = a;
  P.count = a.repetition || a.presence || a.frequency;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DART_F32) e = launch_adjust<float>(P, B, s);
  else if (dtype == DART_F16) e = launch_adjust<__half>(P, B, s);
  else e = launch_adjust<__nv_bfloat16>(P, B, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
