// dart_keep.cu -- what stays in the cache: K8 the walk down a verified tree,
// K9 the rows of a paged cache that are kept, moved up in their order, K10 the
// positions that have gathered the most attention.
//
// K8 (accept_kernel): one CTA per tree.  A node is reached from its parent when
// the parent's pick is its token; every node checks that at once and leaves its
// number at its parent (the lowest wins), then one thread follows the numbers
// from the root: depth + 1 dependent reads of shared memory.  Latency bounds it:
// one round trip to memory, the walk, one store.
//
// K9 (move_kernel): list entry i of a sequence moves position from(i) to base + i,
// from(i) increasing and never below base + i.  So a store of entry i only ever
// hits what an entry j <= i was read from: entries are taken in order, a batch is
// read into registers by the whole CTA, and stored after a barrier.  A CTA owns some
// 16-byte columns of one head of K or V, so no CTA reads what another one writes.
// Columns are dealt to several CTAs (two columns, a 32-byte sector, at least) where
// there are fewer (sequence, head)s than the device can run.  Memory bounds it: two
// passes over the rows that move.
//
// K10 (select_kernel): one CTA per (sequence, head).  The m-th largest score is found
// by a radix search over the ordered keys, 11 + 11 + 10 bits, each level one pass over
// the scores with a histogram in shared memory; a last pass in position order counts
// ties, writes the list and moves the scores up the same way as K9 moves rows.
#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// ------------------------------------------------------------------- accept
struct AcceptParams {
  const int32_t *picks, *tokens, *parents;
  int32_t *path, *counts, *out_tokens;
  int N, depth;
};

__global__ void __launch_bounds__(1024) accept_kernel(const AcceptParams P) {
  __shared__ int32_t pick[kMaxN + 1], next[kMaxN + 1], path[kMaxN + 1];
  __shared__ int count;
  const int b = blockIdx.x, tid = threadIdx.x, N = P.N;
  const int32_t* picks = P.picks + (long long)b * (N + 1);
  // one round trip: a thread's node and its share of the picks are asked for together
  int parent = N, token = -1;
  if (tid < N) {
    parent = P.parents[(long long)b * N + tid];
    token = P.tokens[(long long)b * N + tid];
  }
  for (int i = tid; i <= N; i += blockDim.x) {
    pick[i] = picks[i];
    next[i] = N;
  }
  __syncthreads();
  if (parent >= -1 && parent < tid && token >= 0 && pick[parent + 1] == token) atomicMin(&next[parent + 1], tid);
  __syncthreads();
  if (tid == 0) {
    int at = 0, n = 0;               // row 0 is the root, row i + 1 node i
    path[n++] = 0;
    while (n <= P.depth) {
      const int i = next[at];
      if (i >= N) break;
      at = i + 1;
      path[n++] = at;
    }
    count = n;
    P.counts[b] = n;
  }
  __syncthreads();
  for (int i = tid; i <= P.depth; i += blockDim.x) {
    const bool on = i < count;
    P.path[(long long)b * (P.depth + 1) + i] = on ? path[i] : -1;
    P.out_tokens[(long long)b * (P.depth + 1) + i] = on ? pick[path[i]] : -1;
  }
}

// --------------------------------------------------------------------- move
struct MoveParams {
  dart_cache_t c;
  const int32_t* lengths;
  const int32_t* index;             // [B][heads or 1][width]
  long long index_seq, index_head;  // its strides
  const int32_t* counts;            // [B] entries, or nullptr: min(lengths, width)
  int32_t* out_lengths;             // [B] or nullptr
  int width, relative;              // relative: positions count from lengths[b]
  int cap;                          // positions that a sequence can have
  int slices, vecs;                 // CTAs a row is dealt to, 16-byte columns of each
  FastDiv by_page, by_slices;
  uint32_t* err;
};

constexpr int kMoveUnroll = 4;

__global__ void __launch_bounds__(512) move_kernel(const MoveParams P) {
  const int head = P.by_slices.div(blockIdx.x), slice = blockIdx.x - head * P.slices, b = blockIdx.y;
  const int len = P.lengths[b], cap = P.cap;
  const int32_t* list = P.index + b * P.index_seq + head * P.index_head;
  const int32_t* table = P.c.table + (long long)b * P.c.table_stride;
  const int base = P.relative ? len : 0;
  int count = P.counts ? P.counts[b] : min(len, P.width);
  const bool wrong = len < 0 || count < 0 || count > P.width || len > cap || (P.relative && count > cap - len);
  const bool first = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0;
  if (wrong) {
    if (first) {
      set_dev_error(P.err, DART_DEVERR_CACHE);
      if (P.out_lengths) P.out_lengths[b] = len;
    }
    return;
  }
  if (first && P.out_lengths) P.out_lengths[b] = P.relative ? len + count : count;
  if (!P.relative && count == len) return;          // everything stays where it is
  const long long ps = blockIdx.z ? P.c.v_page_stride : P.c.k_page_stride,
                  rs = blockIdx.z ? P.c.v_row_stride : P.c.k_row_stride,
                  hs = blockIdx.z ? P.c.v_head_stride : P.c.k_head_stride;
  const int all = P.c.dim >> 3;                      // columns of a head
  const int per_row = P.vecs, rows = blockDim.x / per_row;
  const int row = threadIdx.x / per_row, col = slice * per_row + threadIdx.x - row * per_row;
  const bool mine = row < rows && col < all;
  uint16_t* data = static_cast<uint16_t*>(blockIdx.z ? P.c.v : P.c.k) + head * hs + 8 * col;
  auto place = [&](int p) -> uint16_t* {             // nullptr where there is no such position
    if (p < 0 || p >= cap) return nullptr;
    const int at = P.by_page.div(p), page = table[at];
    if (page < 0 || page >= P.c.pages) return nullptr;
    return data + page * ps + (p - at * P.c.page) * rs;
  };
  bool bad = false;
  for (int i0 = 0; i0 < count; i0 += rows * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    uint16_t* to[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + u * rows + row;
      to[u] = nullptr;
      if (!mine || i >= count) continue;
      const int from = list[i], before = i > 0 ? list[i - 1] : -1;
      if (from == i) continue;
      // an entry out of order could be overwritten before it is read: it is left out
      if (from < i || from <= before) {
        bad = true;
        continue;
      }
      const uint16_t* src = from < cap - base ? place(base + from) : nullptr;
      to[u] = place(base + i);
      if (src && to[u]) {
        x[u] = *reinterpret_cast<const uint4*>(src);
      } else {
        to[u] = nullptr;
        bad = true;
      }
    }
    __syncthreads();                                  // the batch is read before any of it is written
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
  if (bad) set_dev_error(P.err, DART_DEVERR_CACHE);
}

// ------------------------------------------------------------------- select
struct SelectParams {
  float* scores;                    // [B][heads][width] with these strides
  long long s_seq, s_head;
  const int32_t* lengths;
  int32_t* index;                   // [B][heads][keep]
  int heads, keep, first, last;
  long long cap;                    // positions of a sequence: the table's and the scores' smaller number
  uint32_t* err;
};

constexpr int kSelectThreads = 1024, kSelectUnroll = 8;

// Larger score, larger key; NaN the least of all.
__device__ __forceinline__ uint32_t score_key(float x) { return x != x ? 0u : ord_f32(x); }

// Exclusive prefix of x over the CTA's threads; total receives the sum.  All threads call it.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();                                   // the sums of the call before have been read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t s = warp_sums[lane];                      // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(kFull, s, 31);
  const uint32_t below = __shfl_sync(kFull, s, warp > 0 ? warp - 1 : 0);
  return incl - x + (warp > 0 ? below : 0u);
}

__global__ void __launch_bounds__(kSelectThreads) select_positions_kernel(const SelectParams P) {
  __shared__ uint32_t bins[2048];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t found[2];
  const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  const int len = P.lengths[b];
  int32_t* out = P.index + ((long long)b * P.heads + h) * P.keep;
  const bool wrong = len < 0 || len > P.cap;
  if (wrong || len <= P.keep) {
    if (wrong && h == 0 && tid == 0) set_dev_error(P.err, DART_DEVERR_CACHE);
    for (int i = tid; i < P.keep; i += kSelectThreads) out[i] = !wrong && i < len ? i : -1;
    return;
  }
  float* scores = P.scores + b * P.s_seq + h * P.s_head;
  const int lo = P.first, hi = len - P.last;          // positions that have to earn their place
  uint32_t want = uint32_t(P.keep - P.first - P.last);
  // want-th largest key: prefix holds its upper bits, found so far
  uint32_t prefix = 0, ties = 0;
  if (want > 0) {
    const int shifts[3] = {21, 10, 0}, sizes[3] = {2048, 2048, 1024};
    for (int level = 0; level < 3; ++level) {
      const int shift = shifts[level], size = sizes[level], above = level == 0 ? 32 : shifts[level - 1];
      for (int i = tid; i < 2048; i += kSelectThreads) bins[i] = 0;
      __syncthreads();
      for (int p0 = lo; p0 < hi; p0 += kSelectThreads * kSelectUnroll) {
        float x[kSelectUnroll];
#pragma unroll
        for (int u = 0; u < kSelectUnroll; ++u) {
          const int p = p0 + u * kSelectThreads + tid;
          x[u] = p < hi ? scores[p] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kSelectUnroll; ++u) {
          const int p = p0 + u * kSelectThreads + tid;
          const uint32_t key = score_key(x[u]);
          if (p < hi && (above == 32 || (key >> above) == prefix)) atomicAdd(&bins[(key >> shift) & (size - 1)], 1u);
        }
      }
      __syncthreads();
      // from the largest bin down: thread t owns bins size - 1 - 2t and the next (one bin each at the last level)
      const int per = size / kSelectThreads;
      uint32_t n[2] = {0u, 0u};
      for (int k = 0; k < per; ++k) n[k] = bins[size - 1 - (tid * per + k)];
      uint32_t total;
      uint32_t at = block_exclusive(n[0] + n[1], warp_sums, total);
      for (int k = 0; k < per; ++k) {
        if (at < want && want <= at + n[k]) {
          found[0] = uint32_t(size - 1 - (tid * per + k));
          found[1] = want - at;
        }
        at += n[k];
      }
      __syncthreads();
      prefix = (prefix << (above - shift)) | found[0];
      want = found[1];
      __syncthreads();
    }
    ties = want;                                     // of the keys equal to prefix, the first `ties` positions stay
  }
  // in position order; the scores move up behind those that were read before them
  uint32_t kept = 0, seen = 0;
  for (int p0 = 0; p0 < len; p0 += kSelectThreads) {
    const int p = p0 + tid;
    const float x = p < len ? scores[p] : 0.f;
    const uint32_t key = score_key(x);
    const bool free = p >= lo && p < hi;
    const bool sure = p < len && (!free || (ties > 0 && key > prefix));
    const bool tie = free && ties > 0 && key == prefix;
    // both counts in one word: a batch holds at most 1024 of either
    uint32_t total;
    const uint32_t before = block_exclusive((sure ? 1u : 0u) | (tie ? 1u << 16 : 0u), warp_sums, total);
    const uint32_t tie_rank = seen + (before >> 16);
    const uint32_t ties_before = min(tie_rank, ties) - min(seen, ties);
    if (sure || (tie && tie_rank < ties)) {
      const uint32_t i = kept + (before & 0xFFFFu) + ties_before;
      out[i] = p;
      scores[i] = x;
    }
    kept += (total & 0xFFFFu) + min(seen + (total >> 16), ties) - min(seen, ties);
    seen += total >> 16;
  }
  __syncthreads();
  for (int p = P.keep + tid; p < len; p += kSelectThreads) scores[p] = 0.f;
}

cudaError_t launch_move(MoveParams& P, int B, cudaStream_t s) {
  // A row's columns are dealt to several CTAs until there are about two for each SM; at
  // least two columns each, so that whole 32-byte sectors move.
  const int all = P.c.dim / 8, sms = device_sms() > 0 ? device_sms() : 152;
  int vecs = all;
  while (vecs > 2 && 2ll * B * P.c.heads * ((all + vecs - 1) / vecs) < 2ll * sms) vecs = (vecs + 1) / 2;
  P.vecs = vecs;
  P.slices = (all + vecs - 1) / vecs;
  P.by_slices = fast_div(uint32_t(P.slices));
  P.by_page = fast_div(uint32_t(P.c.page));
  // as many threads as the list can use
  long long threads = (long long)((P.width + kMoveUnroll - 1) / kMoveUnroll) * vecs;
  threads = threads > 512 ? 512 : (threads + 31) / 32 * 32;
  return launch_kernel(move_kernel, dim3(unsigned(P.c.heads * P.slices), unsigned(B), 2), dim3(unsigned(threads)), 0, s, P);
}

}  // namespace
}  // namespace dart

extern "C" int dart_tree_accept(const int32_t* picks, const int32_t* tokens, const int32_t* parents, int B, int N,
                                int depth, int32_t* out_path, int32_t* out_counts, int32_t* out_tokens, void* stream) {
  using namespace dart;
  if (B < 0 || N < 0 || N > kMaxN || depth < 0 || depth > N) return DART_ERR_INVALID_ARG;
  if (B == 0) return DART_OK;
  if (!picks || !out_path || !out_counts || !out_tokens || (N > 0 && (!tokens || !parents))) return DART_ERR_INVALID_ARG;
  const AcceptParams P{picks, tokens, parents, out_path, out_counts, out_tokens, N, depth};
  const int threads = N < 32 ? 32 : (N + 31) / 32 * 32;
  const cudaError_t e = launch_kernel(accept_kernel, unsigned(B), unsigned(threads), 0, static_cast<cudaStream_t>(stream), P);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}

extern "C" int dart_kv_keep(const dart_cache_t* cache, const int32_t* lengths, const int32_t* path, int64_t path_stride,
                            const int32_t* counts, int B, int width, int32_t* out_lengths, uint32_t* device_err,
                            void* stream) {
  using namespace dart;
  if (B < 0 || B > 65535 || width < 1 || width > (1 << 30)) return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (path_stride < 0 || (B > 1 && path_stride < width)) return DART_ERR_INVALID_ARG;
  if (B == 0) return DART_OK;
  if (!lengths || !path || !counts || cache->pages < 1 || cache->table_width < 1) return DART_ERR_INVALID_ARG;
  MoveParams P;
  P.c = *cache;
  P.lengths = lengths;
  P.index = path; P.index_seq = path_stride; P.index_head = 0;
  P.counts = counts;
  P.out_lengths = out_lengths;
  P.width = width; P.relative = 1;
  P.cap = cache->table_width * cache->page;
  P.err = device_err;
  return launch_move(P, B, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}

extern "C" int dart_kv_evict(const dart_cache_t* cache, const int32_t* lengths, int B, float* scores,
                             int64_t scores_seq_stride, int64_t scores_head_stride, int scores_width, int keep,
                             int first, int last, int32_t* out_index, int32_t* out_lengths, uint32_t* device_err,
                             void* stream) {
  using namespace dart;
  if (B < 0 || B > 65535 || scores_width < 0 || keep < 1 || first < 0 || last < 0 || first > keep || last > keep - first)
    return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (scores_seq_stride < 0 || scores_head_stride < 0 || (cache->heads > 1 && scores_head_stride < scores_width) ||
      (B > 1 && scores_seq_stride < scores_width))
    return DART_ERR_INVALID_ARG;
  if (B == 0) return DART_OK;
  if (!lengths || !scores || !out_index || cache->pages < 1 || cache->table_width < 1) return DART_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long cap = (long long)cache->table_width * cache->page;
  SelectParams S;
  S.scores = scores; S.s_seq = scores_seq_stride; S.s_head = scores_head_stride;
  S.lengths = lengths; S.index = out_index; S.heads = cache->heads;
  S.keep = keep; S.first = first; S.last = last;
  S.cap = cap < scores_width ? cap : scores_width;
  S.err = device_err;
  cudaError_t e = launch_kernel(select_positions_kernel, dim3(unsigned(cache->heads), unsigned(B)), kSelectThreads, 0, s, S);
  if (e != cudaSuccess) return DART_ERR_CUDA;
  MoveParams P;
  P.c = *cache;
  P.lengths = lengths;
  P.index = out_index; P.index_seq = (long long)cache->heads * keep; P.index_head = keep;
  P.counts = nullptr;
  P.out_lengths = out_lengths;
  P.width = keep; P.relative = 0;
  P.cap = int(S.cap);
  P.err = device_err;
  return launch_move(P, B, s) == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
