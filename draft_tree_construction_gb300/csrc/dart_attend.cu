// dart_attend.cu -- K7: attention of a chunk of new tokens over a paged cache,
// the chunk's tail being a tree with packed ancestor-or-self masks.
//
// One CTA per token and query head: 128 positions at a time, a thread each for
// the scores, a running maximum and sum, then a thread per output element.
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 128;

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  long long q_ts, q_hs, o_ts, o_hs;
  int Hq, Hkv, G, D, T, B, N;
  const int32_t* lengths;
  const int32_t* starts;
  const uint32_t* mask;
  float scale;
  dart_cache_t c;
  uint32_t* err;
};

template <typename T> __device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kThreads)
attend_kernel(const AttendParams P) {
  __shared__ float sq[128];
  __shared__ float sp[kThreads];
  __shared__ int spage[kThreads];
  __shared__ float red[4];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  const dart_cache_t& C = P.c;
  int b = 0;
  while (b < P.B && P.starts[b + 1] <= t) ++b;
  if (b >= P.B || P.starts[b] > t) return;
  const int i = t - P.starts[b], n = min(P.starts[b + 1], P.T) - P.starts[b];
  const int len = max(P.lengths[b], 0);
  const long long cap = (long long)C.table_width * C.page;
  long long S = (long long)len + n;
  if (S > cap || P.lengths[b] < 0) {
    if (tid == 0) set_dev_error(P.err, DART_DEVERR_CACHE);
    if (S > cap) S = cap;
  }
  const int lead = max(n - P.N, 0);
  const long long plain = (long long)len + (i < lead ? i + 1 : lead);   // positions below are visible
  const long long end = i < lead ? min(plain, S) : S;
  const int MW = (P.N + 31) / 32;
  const uint32_t* bits = i >= lead ? P.mask + ((long long)b * P.N + (i - lead)) * MW : nullptr;

  const int hk = h / P.G;
  const T* q = static_cast<const T*>(P.q) + (long long)t * P.q_ts + (long long)h * P.q_hs;
  if (tid < P.D) sq[tid] = to_float(q[tid]) * P.scale;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (long long p0 = 0; p0 < end; p0 += kThreads) {
    const long long p = p0 + tid;
    float s = -INFINITY;
    int page = -1;
    __syncthreads();
    if (p < end) {
      bool see = p < plain;
      if (!see && bits) {
        const int j = int(p - plain);
        see = j < P.N && ((bits[j >> 5] >> (j & 31)) & 1u);
      }
      if (see) {
        page = C.table[(long long)b * C.table_stride + p / C.page];
        if (page < 0 || page >= C.pages) {
          set_dev_error(P.err, DART_DEVERR_CACHE);
          page = -1;
        }
        s = 0.f;
        if (page >= 0) {
          const T* k = static_cast<const T*>(C.k) + page * C.k_page_stride + (p % C.page) * C.k_row_stride +
                       (long long)hk * C.k_head_stride;
          for (int d = 0; d < P.D; ++d) s += sq[d] * to_float(k[d]);
        }
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    if (lane == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    if (mn == -INFINITY) continue;
    const float keep = expf(m - mn);
    const float e = expf(s - mn);
    m = mn;
    float sum = e;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sp[tid] = e;
    spage[tid] = page;
    __syncthreads();
    if (lane == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * keep + (red[0] + red[1] + red[2] + red[3]);
    acc *= keep;
    if (tid < P.D)
      for (int j = 0; j < kThreads; ++j)
        if (spage[j] >= 0)
          acc += sp[j] * to_float(static_cast<const T*>(C.v)[spage[j] * C.v_page_stride +
                                                             ((p0 + j) % C.page) * C.v_row_stride +
                                                             (long long)hk * C.v_head_stride + tid]);
  }
  if (tid < P.D)
    (static_cast<T*>(P.out) + (long long)t * P.o_ts + (long long)h * P.o_hs)[tid] =
        from_float<T>(l > 0.f ? acc / l : 0.f);
  if (P.lse && tid == 0) P.lse[(long long)t * P.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

bool mult8(long long a, long long b) { return ((a | b) & 7) == 0; }
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace dart

extern "C" size_t dart_attention_workspace_bytes(int T, int B, int q_heads, int heads, int dim) {
  if (T < 0 || B < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || dim < 8 || dim > 128 || dim % 8 != 0)
    return 0;
  return dart::kCtrlBytes;
}

extern "C" int dart_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                                   int T, int B, const int32_t* lengths, const int32_t* starts,
                                   const uint32_t* mask, int N, float scale, const dart_cache_t* cache,
                                   void* out, int64_t out_token_stride, int64_t out_head_stride, float* out_lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dart;
  if (T < 0 || T > (1 << 26) || B < 0 || q_heads < 1 || q_heads > 65535 || N < 0 || N > kMaxN)
    return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (q_heads % cache->heads != 0 || !std::isfinite(scale)) return DART_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DART_OK;
  if (!aligned16(q) || !aligned16(out) || !mult8(q_token_stride, q_head_stride) ||
      !mult8(out_token_stride, out_head_stride) || !lengths || !starts || (N > 0 && !mask))
    return DART_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 ||
      workspace_bytes < dart_attention_workspace_bytes(T, B, q_heads, cache->heads, cache->dim))
    return DART_ERR_WORKSPACE;
  AttendParams P;
  P.q = q; P.out = out; P.lse = out_lse;
  P.q_ts = q_token_stride; P.q_hs = q_head_stride;
  P.o_ts = out_token_stride; P.o_hs = out_head_stride;
  P.Hq = q_heads; P.Hkv = cache->heads; P.G = q_heads / cache->heads; P.D = cache->dim;
  P.T = T; P.B = B; P.N = N;
  P.lengths = lengths; P.starts = starts; P.mask = mask; P.scale = scale;
  P.c = *cache;
  P.err = static_cast<uint32_t*>(workspace);
  const dim3 grid(T, q_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cache->dtype == DART_F16) attend_kernel<__half><<<grid, kThreads, 0, s>>>(P);
  else attend_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
