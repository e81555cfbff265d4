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
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjWarpTokens = 1024;                       // tokens of the slice that one warp owns
constexpr int kAdjSlice = kAdjWarps * kAdjWarpTokens;      // tokens per CTA
constexpr int kAdjWords = kAdjSlice / 32;
constexpr int kMaxBias = 1024;                             // biases per sequence
constexpr unsigned kFull = 0xFFFFFFFFu;

struct AdjustParams {
  const void* in;
  void* out;
  int R, V, row_group;                 // rows per CTA
  long long in_stride, out_stride;
  dart_adjust_t a;
  bool count;                          // some penalty is given
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

// `count` (<= 32) bits from bit `at` on of a word array of `words` words.
__device__ __forceinline__ uint32_t bits_at(const uint32_t* w, int at, int words) {
  const int i = at >> 5;
  const uint32_t lo = w[i];
  if ((at & 31) == 0) return lo;
  const uint32_t hi = i + 1 < words ? w[i + 1] : 0u;
  return __funnelshift_r(lo, hi, at & 31);
}

template <typename T>
__global__ void __launch_bounds__(kAdjThreads)
adjust_kernel(const AdjustParams P) {
  constexpr int E = 16 / int(sizeof(T));
  extern __shared__ __align__(16) unsigned char smem[];
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem);                         // [kAdjSlice]
  float* bias = reinterpret_cast<float*>(smem) + (P.count ? kAdjSlice : 0);     // [kAdjSlice]
  __shared__ uint32_t cnt_bits[kAdjWords + 1];     // token is counted
  __shared__ uint32_t bias_bits[kAdjWords + 1];    // token has a bias
  __shared__ int32_t list_id[kMaxBias];            // the slice's biases, in their order
  __shared__ int32_t warp_n[kAdjWarps];

  const int b = blockIdx.z;
  const int v0 = blockIdx.x * kAdjSlice;
  const int vn = min(P.V - v0, kAdjSlice);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const dart_adjust_t& a = P.a;

  for (int i = tid; i <= kAdjWords; i += kAdjThreads) cnt_bits[i] = bias_bits[i] = 0u;
  if (P.count)
    for (int i = tid; i < kAdjSlice; i += kAdjThreads) counts[i] = 0u;
  __syncthreads();
  if (P.count && a.history) {
    const int32_t* h = a.history + (long long)b * a.history_stride;
    const int len = a.history_len ? max(0, min(a.history_len[b], a.history_width)) : a.history_width;
    for (int i = tid; i < len; i += kAdjThreads) {
      const uint32_t t = uint32_t(h[i]) - uint32_t(v0);
      if (t < uint32_t(vn)) {
        atomicAdd(&counts[t], 1u);
        atomicOr(&cnt_bits[t >> 5], 1u << (t & 31));
      }
    }
  }
  if (a.bias_count > 0) {
    // The slice's biases, compacted in their order; then the first entry of
    // each id sums that id's values in order, so that repeated ids always give
    // the same sum.
    __shared__ float list_val[kMaxBias];
    int n = 0;
    for (int base = 0; base < a.bias_count; base += kAdjThreads) {
      const int i = base + tid;
      uint32_t t = kFull;
      if (i < a.bias_count) t = uint32_t(a.bias_ids[(long long)b * a.bias_count + i]) - uint32_t(v0);
      const bool in = t < uint32_t(vn);
      const unsigned m = __ballot_sync(kFull, in);
      if (lane == 0) warp_n[warp] = __popc(m);
      __syncthreads();
      int at = n + __popc(m & ((1u << lane) - 1u));
      for (int w = 0; w < kAdjWarps; ++w) {
        if (w < warp) at += warp_n[w];
        n += warp_n[w];
      }
      if (in) {
        list_id[at] = int32_t(t);
        list_val[at] = a.bias_vals[(long long)b * a.bias_count + i];
      }
      __syncthreads();
    }
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
    }
  }
  __syncthreads();

  // from here on a warp touches its own tokens only
  const int w0 = warp * kAdjWarpTokens;
  const int wn = min(vn - w0, kAdjWarpTokens);
  if (wn <= 0) return;
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const int words = (P.V + 31) >> 5;
  const int MW = (a.N + 31) >> 5;
  const int r_end = min(P.R, int(blockIdx.y + 1) * P.row_group);

  // the counted / biased element t (index within the slice)
  auto adjusted = [&](T raw, int t) -> T {
    float x = Elem<T>::get(raw);
    if ((cnt_bits[t >> 5] >> (t & 31)) & 1u) {
      const uint32_t c = counts[t];
      x = x > 0.f ? x / rep : x * rep;
      x = x - freq * float(c) - pres;
    }
    if ((bias_bits[t >> 5] >> (t & 31)) & 1u) x += bias[t];
    return Elem<T>::put(x);
  };

  for (int r = blockIdx.y * P.row_group; r < r_end; ++r) {
    const long long row = (long long)b * P.R + r;
    const T* in = static_cast<const T*>(P.in) + row * P.in_stride + v0;
    T* out = static_cast<T*>(P.out) + row * P.out_stride + v0;
    const uint32_t* allow =
        a.allowed ? a.allowed + (long long)b * a.allowed_seq_stride + (long long)r * a.allowed_row_stride : nullptr;

    // the tokens on this row's path that the warp owns join the counts
    const int node = r - (P.R - a.N);
    const bool path = P.count && a.N > 0 && node >= 0;
    uint32_t on_path = 0;
    const int32_t* toks = nullptr;
    if (path) {
      toks = a.tokens + (long long)b * a.N + 32 * lane;
      if (lane < MW) {
        on_path = a.mask[((long long)b * a.N + node) * MW + lane];
        if (32 * lane + 32 > a.N) on_path &= (1u << (a.N & 31)) - 1u;
      }
      for (uint32_t m = on_path; m; m &= m - 1) {
        const uint32_t t = uint32_t(toks[__ffs(m) - 1]) - uint32_t(v0 + w0);
        if (t < uint32_t(wn)) {
          atomicAdd(&counts[w0 + t], 1u);
          atomicOr(&cnt_bits[(w0 + t) >> 5], 1u << (t & 31));
        }
      }
      __syncwarp();
    }

    auto scalar = [&](int t) {
      const uint32_t word = allow ? allow[(v0 + t) >> 5] : kFull;
      T x;
      if ((word >> ((v0 + t) & 31)) & 1u) {
        x = in[t];
        if (((cnt_bits[t >> 5] | bias_bits[t >> 5]) >> (t & 31)) & 1u) x = adjusted(x, t);
      } else {
        x = Elem<T>::put(-INFINITY);
      }
      out[t] = x;
    };
    // elements before the first 16-byte boundary of the warp's part
    const int phase = int((reinterpret_cast<uintptr_t>(in + w0) / sizeof(T)) % E);
    const int head = min((E - phase) % E, wn);
    if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0) {
      const int nv = (wn - head) / E;
      for (int i = lane; i < nv; i += 32) {
        const int t = w0 + head + i * E;
        constexpr uint32_t all = (1u << E) - 1u;
        const uint32_t ok = (allow ? bits_at(allow, v0 + t, words) : kFull) & all;
        Vec<T> x;
        if (ok == 0u) {
          x.u = make_uint4(Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf, Elem<T>::kNegInf);
        } else {
          x.u = *reinterpret_cast<const uint4*>(in + t);
          const uint32_t hit = (bits_at(cnt_bits, t, kAdjWords + 1) | bits_at(bias_bits, t, kAdjWords + 1)) & all;
          if (hit & ok) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if ((hit >> e) & 1u) x.e[e] = adjusted(x.e[e], t + e);
          }
          if (ok != all) {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (!((ok >> e) & 1u)) x.e[e] = Elem<T>::put(-INFINITY);
          }
        }
        *reinterpret_cast<uint4*>(out + t) = x.u;
      }
      if (lane < head) scalar(w0 + lane);
      const int tail = head + nv * E;
      if (lane < wn - tail) scalar(w0 + tail + lane);
    } else {
      for (int i = lane; i < wn; i += 32) scalar(w0 + i);
    }

    if (path) {        // and leave them again
      __syncwarp();
      for (uint32_t m = on_path; m; m &= m - 1) {
        const uint32_t t = uint32_t(toks[__ffs(m) - 1]) - uint32_t(v0 + w0);
        if (t < uint32_t(wn)) {
          if (atomicSub(&counts[w0 + t], 1u) == 1u) atomicAnd(&cnt_bits[(w0 + t) >> 5], ~(1u << (t & 31)));
        }
      }
      __syncwarp();
    }
  }
}

template <typename T>
cudaError_t launch_adjust(const AdjustParams& P, dim3 grid, size_t smem, cudaStream_t stream) {
  const cudaError_t e =
      cudaFuncSetAttribute(adjust_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kAdjSlice);
  if (e != cudaSuccess) return e;
  adjust_kernel<T><<<grid, kAdjThreads, smem, stream>>>(P);
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
  const int slices = (V + kAdjSlice - 1) / kAdjSlice;
  // rows per CTA: enough CTAs to fill the device a few times, then as many rows
  // as possible share one count
  const long long want = 152ll * 3 * 4;
  const long long per = (long long)slices * B;
  long long groups = (want + per - 1) / per;
  groups = groups < 1 ? 1 : groups > R ? R : groups;
  if (groups > 65535) groups = 65535;
  P.row_group = int((R + groups - 1) / groups);
  const dim3 grid(slices, (R + P.row_group - 1) / P.row_group, B);
  const size_t smem = size_t(4 * kAdjSlice) * ((P.count ? 1 : 0) + (a.bias_count > 0 ? 1 : 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DART_F32) e = launch_adjust<float>(P, grid, smem, s);
  else if (dtype == DART_F16) e = launch_adjust<__half>(P, grid, smem, s);
  else e = launch_adjust<__nv_bfloat16>(P, grid, smem, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
