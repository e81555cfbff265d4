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
// read into registers by the whole CTA, and stored after a barrier.  A CTA, or a cluster
// of up to eight with a barrier of its own where lists are long and heads few, has one head
// of K or V, so nobody reads what another one writes.  A lane finds where one of the
// warp's 32 rows lies; then the warp moves them, whole rows at a time (when each thread
// found its own 16 bytes, that was 150 instructions for each, and they bound it).  Memory
// bounds it: two passes over the rows that move.  What the positions have gathered goes with
// them in one more layer of the grid, a CTA a head.
//
// K10 (select_kernel): the m-th largest score is found by a radix search over the
// ordered keys, 11 + 11 + 10 bits.  One CTA per (sequence, head), or a cluster of up to
// eight that share its positions where there are few or long ones.  A CTA reads its scores
// once, into registers; each level is a histogram in shared memory, which the cluster's
// CTAs read from one another, and a scan.  Then every warp counts what it keeps by ballots,
// one scan gives all places, and the list and the scores, which have all been read by then,
// are written.  Latency bounds it.  Where the page table and the scores have room for more than
// registers hold (163840 positions a head), whatever the lengths are, one CTA a head reads them
// again at every level (long_kernel).
//
// Measured (GB300, graph-replayed): a tree walked and its path moved, 8 heads of 128, 6.4 us
// for one tree of 78 nodes, 8.4 for 64 of 496 (two launches).  Eviction of fresh scores: 32
// sequences of about 6000 positions to 2048, 105 us, 80 of them the moves (6.7 TB/s); one of
// 32768 to 16384, 50 us: 20 the selection (eight cluster barriers in a chain: two a level, one before
// the places, one at the end), 30 the moves of 128 CTAs (4.5 TB/s).  Where hardly any row moves: 36 and
// 28.  A path's scores moved and cleared with its rows add nothing to the 4.1 and 6.2 us of the move.
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
  int ranks;                        // CTAs that share a head's list
  // what each position has gathered, moved with it by the CTAs of grid layer `scored` (-1: none)
  int scored, s_width;
  float* scores;
  long long s_seq, s_head;
  const int32_t* starts;            // [B + 1]: the chunk's end
  FastDiv by_page;
  uint32_t* err;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMoveThreads = 256;

// Whether entry i, `from`, may be moved: one out of order could be overwritten before it is read, or
// name a row that another entry has.  before: the entry in front of it, -1 for the first.
__device__ __forceinline__ bool in_order(int from, int before, int i, int end) {
  return from >= i && from > before && from < end;
}

// The scores of one head, by one CTA: those of the list's positions move up as the rows do, those from
// there to the chunk's end become 0, so that the next chunk's positions begin with nothing.
__device__ __forceinline__ void move_scores(const MoveParams& P, const int32_t* list, int b, int head, int base, int count) {
  const int tid = threadIdx.x, threads = blockDim.x;
  float* row = P.scores + b * P.s_seq + head * P.s_head;
  const long long end = (long long)base + ((long long)P.starts[b + 1] - P.starts[b]);
  bool bad = end > P.s_width;
  for (int i0 = 0; i0 < count; i0 += threads) {
    const int i = i0 + tid, from = i < count ? list[i] : i, before = i < count && i > 0 ? list[i - 1] : -1;
    bool moves = from != i;
    if (i < count && !in_order(from, before, i, P.cap - base)) {
      bad = true;
      moves = false;
    }
    if (moves && base + from >= P.s_width) bad = true;         // has no score: what it leaves is 0
    const float x = moves && base + from < P.s_width ? row[base + from] : 0.f;
    __syncthreads();                                           // as for the rows: a batch is read before it is written
    if (moves && base + i < P.s_width) row[base + i] = x;
  }
  const int stop = int(max(min(end, (long long)P.s_width), 0ll));
  for (int p = base + count + tid; p < stop; p += threads) row[p] = 0.f;
  if (bad) set_dev_error(P.err, DART_DEVERR_CACHE);
}

// COLS: 16-byte columns of a row, rounded up to a power of two; a warp moves 32 / COLS rows at once.
template <int COLS>
__global__ void __launch_bounds__(kMoveThreads, 2) move_kernel(const MoveParams P) {
  const int head = int(blockIdx.x) / P.ranks, rank = int(blockIdx.x) - head * P.ranks, b = blockIdx.y;
  const int len = P.lengths[b], cap = P.cap;
  const int32_t* list = P.index + b * P.index_seq + head * P.index_head;
  const int32_t* table = P.c.table + (long long)b * P.c.table_stride;
  const int base = P.relative ? len : 0;
  const int count = P.counts ? P.counts[b] : min(len, P.width);
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
  if (int(blockIdx.z) == P.scored) {
    if (rank == 0) move_scores(P, list, b, head, base, count);
    return;
  }
  if (!P.relative && count == len) return;          // everything stays where it is
  const long long ps = blockIdx.z ? P.c.v_page_stride : P.c.k_page_stride,
                  rs = blockIdx.z ? P.c.v_row_stride : P.c.k_row_stride,
                  hs = blockIdx.z ? P.c.v_head_stride : P.c.k_head_stride;
  constexpr int kRows = 32 / COLS;                   // rows of a step, COLS steps for the warp's 32
  const int lane = threadIdx.x & 31, warps = int(blockDim.x) >> 5, warp = int(threadIdx.x) >> 5;
  const int sub = lane / COLS, col = lane % COLS;
  const bool mine = col < (P.c.dim >> 3);
  uint4* data = reinterpret_cast<uint4*>(static_cast<uint16_t*>(blockIdx.z ? P.c.v : P.c.k) + head * hs) + col;
  // where position p's row begins, in 16-byte units from the head's first; -1 where there is none
  auto place = [&](int p, int page) -> long long {
    if (page < 0 || page >= P.c.pages) return -1;
    return (page * ps + (p - P.by_page.div(p) * P.c.page) * rs) >> 3;
  };
  bool bad = false;
  const int stride = 32 * warps * P.ranks;           // entries of a batch
  int next = (rank * warps + warp) * 32 + lane;      // this lane's entry
  int from = next < count ? list[next] : next, before = next < count && next > 0 ? list[next - 1] : -1;
  for (int i0 = 0; i0 < count; i0 += stride) {
    const int i = next;
    bool moves = from != i;
    if (i < count && !in_order(from, before, i, cap - base)) {
      bad = true;
      moves = false;
    }
    long long src = -1, dst = -1;
    if (moves) {
      const int s = base + from, d = base + i, s_page = table[P.by_page.div(s)], d_page = table[P.by_page.div(d)];
      src = place(s, s_page);
      dst = place(d, d_page);
      if (src < 0 || dst < 0) {
        bad = true;
        src = dst = -1;
      }
    }
    // the next batch's entry is on its way meanwhile
    next += stride;
    from = next < count ? list[next] : next;
    before = next < count ? list[next - 1] : -1;
    const bool any = __any_sync(kFull, src >= 0);
    uint4 x[COLS];
    if (any) {
#pragma unroll
      for (int u = 0; u < COLS; ++u) {
        const long long at = __shfl_sync(kFull, src, u * kRows + sub);
        if (at >= 0 && mine) x[u] = data[at];
      }
    }
    // the batch is read before any of it is written
    if (P.ranks > 1) cluster_sync();
    else __syncthreads();
    if (any) {
#pragma unroll
      for (int u = 0; u < COLS; ++u) {
        const long long at = __shfl_sync(kFull, dst, u * kRows + sub);
        if (at >= 0 && mine) data[at] = x[u];
      }
    }
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

__global__ void __launch_bounds__(kSelectThreads) long_kernel(const SelectParams P) {
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

// ---- a cluster's CTAs, a head's scores in their registers
__device__ __forceinline__ uint32_t load_there(const uint32_t* p, uint32_t rank) {
  uint32_t at, x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

// Four words at once.
__device__ __forceinline__ uint4 load_four_there(const uint32_t* p, uint32_t rank) {
  uint32_t at;
  uint4 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
  return x;
}

__device__ __forceinline__ void store_four_there(const uint32_t* p, uint32_t rank, const uint4& x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1,%2,%3,%4};" :: "r"(at), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

constexpr int kShareThreads = 512, kShareWarps = kShareThreads / 32, kMaxRanks = 8;

// Exclusive prefix over 512 threads; total receives the sum.
__device__ __forceinline__ uint32_t share_exclusive(uint32_t x, uint32_t* warp_sums, uint32_t& total) {
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
  uint32_t below = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kShareWarps; ++w) {
    if (w == warp) below = total;
    total += warp_sums[w];
  }
  return below + incl - x;
}

template <int KEYS>
__global__ void __launch_bounds__(kShareThreads, KEYS <= 20 ? 2 : 1) select_kernel(const SelectParams P, int ranks) {
  __shared__ alignas(16) uint32_t bins[2][2048];     // of a level and the next, which is cleared while others read the first
  __shared__ alignas(16) uint32_t sums[2048];        // a cluster's bins together
  __shared__ uint32_t warp_sums[kShareWarps];
  __shared__ uint32_t found[2], kept_here[2];
  __shared__ uint32_t counts[KEYS * kShareWarps];    // kept below 16, ties above, of each batch and warp
  const int rank = int(blockIdx.x) % ranks, h = int(blockIdx.x) / ranks, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = P.lengths[b];
  int32_t* out = P.index + ((long long)b * P.heads + h) * P.keep;
  const bool wrong = len < 0 || len > P.cap;
  if (wrong || len <= P.keep) {
    if (wrong && blockIdx.x == 0 && tid == 0) set_dev_error(P.err, DART_DEVERR_CACHE);
    for (int i = rank * kShareThreads + tid; i < P.keep; i += ranks * kShareThreads) out[i] = !wrong && i < len ? i : -1;
    return;
  }
  float* scores = P.scores + b * P.s_seq + h * P.s_head;
  const int lo = P.first, hi = len - P.last;          // positions that have to earn their place
  // this CTA's positions, in batches of 512
  const int share = (len + ranks - 1) / ranks, p0 = min(rank * share, len), p1 = min(p0 + share, len);
  float x[KEYS];
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const int p = p0 + i * kShareThreads + tid;
    x[i] = p < p1 ? scores[p] : 0.f;
  }
  for (int i = tid; i < 2048; i += kShareThreads) bins[0][i] = 0;
  uint32_t want = uint32_t(P.keep - P.first - P.last), prefix = 0, ties = 0;
  if (want > 0) {
    const int shifts[3] = {21, 10, 0}, sizes[3] = {2048, 2048, 1024};
#pragma unroll
    for (int level = 0; level < 3; ++level) {
      const int shift = shifts[level], size = sizes[level], above = level == 0 ? 32 : shifts[level - 1];
      uint32_t* here = bins[level & 1];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < KEYS; ++i) {
        if (p0 + i * kShareThreads >= p1) break;
        const int p = p0 + i * kShareThreads + tid;
        const uint32_t key = score_key(x[i]);
        const bool on = p < p1 && p >= lo && p < hi && (level == 0 || (key >> (above & 31)) == prefix);
        const uint32_t bin = (key >> shift) & (size - 1), who = __ballot_sync(kFull, on);
        if (who == 0) continue;
        // scores that got nothing yet are equal: then one add for the warp
        const uint32_t first = __shfl_sync(kFull, bin, __ffs(who) - 1);
        if (__all_sync(kFull, !on || bin == first)) {
          if (lane == 0) atomicAdd(&here[first], uint32_t(__popc(who)));
        } else if (on) {
          atomicAdd(&here[bin], 1u);
        }
      }
      if (ranks > 1) cluster_sync();
      else __syncthreads();
      // A cluster's CTAs each add up their part of the bins over all of them and hand the sums to
      // all (when each added up all bins for itself, a level took twice as long).
      if (ranks > 1) {
        const int part = 2048 / ranks, first = rank * part;
        for (int i = 4 * tid; i < part; i += 4 * kShareThreads) {
          uint4 all = make_uint4(0, 0, 0, 0), from[kMaxRanks];
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r)
            if (r < ranks) from[r] = load_four_there(&here[first + i], uint32_t(r));
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r)
            if (r < ranks) all = make_uint4(all.x + from[r].x, all.y + from[r].y, all.z + from[r].z, all.w + from[r].w);
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r)
            if (r < ranks) store_four_there(&sums[first + i], uint32_t(r), all);
        }
        cluster_sync();
      }
      // from the largest bin down: thread t owns the four from 2047 - 4 t on
      const uint4 four = *reinterpret_cast<const uint4*>(&(ranks > 1 ? sums : here)[2044 - 4 * tid]);
      const uint32_t n[4] = {four.w, four.z, four.y, four.x}, sum = four.x + four.y + four.z + four.w;
      if (level < 2)
        for (int i = tid; i < 2048; i += kShareThreads) bins[(level + 1) & 1][i] = 0;
      uint32_t total;
      uint32_t at = share_exclusive(sum, warp_sums, total);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at < want && want <= at + n[k]) {
          found[0] = uint32_t(2047 - (tid * 4 + k));
          found[1] = want - at;
        }
        at += n[k];
      }
      __syncthreads();
      prefix = level == 0 ? found[0] : (prefix << (above - shift)) | found[0];
      want = found[1];
    }
    ties = want;                                     // of the keys equal to prefix, the first `ties` positions stay
  }
  // what each warp keeps of each batch
  auto sure_of = [&](int p, uint32_t key) { return p < p1 && (p < lo || p >= hi || (ties > 0 && key > prefix)); };
  auto tie_of = [&](int p, uint32_t key) { return p < p1 && p >= lo && p < hi && ties > 0 && key == prefix; };
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    if (p0 + i * kShareThreads >= p1) {
      if (lane == 0) counts[i * kShareWarps + warp] = 0;
      continue;
    }
    const int p = p0 + i * kShareThreads + tid;
    const uint32_t key = score_key(x[i]);
    const uint32_t sure = __ballot_sync(kFull, sure_of(p, key)), tie = __ballot_sync(kFull, tie_of(p, key));
    if (lane == 0) counts[i * kShareWarps + warp] = uint32_t(__popc(sure)) | uint32_t(__popc(tie)) << 16;
  }
  __syncthreads();
  // places of the batches' warps: both sums of at most 20480 in one word
  constexpr int kEach = (KEYS * kShareWarps + kShareThreads - 1) / kShareThreads;
  uint32_t own[kEach], sum = 0, total;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid * kEach + e;
    own[e] = i < KEYS * kShareWarps ? counts[i] : 0u;
    sum += own[e];
  }
  uint32_t at = share_exclusive(sum, warp_sums, total);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = tid * kEach + e;
    if (i < KEYS * kShareWarps) counts[i] = at;
    at += own[e];
  }
  if (tid == 0) kept_here[0] = total;
  uint32_t kept = 0, seen = 0;                       // before this CTA's positions
  if (ranks > 1) {
    cluster_sync();                                  // and every score has been read
    for (int r = 0; r < rank; ++r) {
      const uint32_t t = load_there(&kept_here[0], uint32_t(r));
      kept += t & 0xFFFFu;
      seen += t >> 16;
    }
  } else {
    __syncthreads();
  }
  kept += min(seen, ties);
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    if (p0 + i * kShareThreads >= p1) break;
    const int p = p0 + i * kShareThreads + tid;
    const uint32_t key = score_key(x[i]);
    const bool sure = sure_of(p, key), tie = tie_of(p, key);
    const uint32_t below = (1u << lane) - 1u, before = counts[i * kShareWarps + warp];
    const uint32_t sures = __popc(__ballot_sync(kFull, sure) & below), tied = __popc(__ballot_sync(kFull, tie) & below);
    const uint32_t tie_rank = seen + (before >> 16) + tied;
    if (sure || (tie && tie_rank < ties)) {
      const uint32_t to = kept + (before & 0xFFFFu) + sures + min(tie_rank, ties) - min(seen, ties);
      out[to] = p;
      scores[to] = x[i];
    }
  }
  // what lies behind the kept ones: nobody's place, so no order matters
  for (int p = max(p0, P.keep) + tid; p < p1; p += kShareThreads) scores[p] = 0.f;
  if (ranks > 1) cluster_sync();                     // the others have read this CTA's words
}

cudaError_t launch_select(const SelectParams& S, int B, cudaStream_t s) {
  // As many CTAs a head as its positions need, and up to two an SM in all while each has
  // 2048 positions at least; the moves below likewise (both together, with and without: one
  // sequence of 32768 to 16384, 8 heads 48 us for 127, one head 35 for 119; 4 of 8192 to 4096 34 for 45).
  // Lengths are on the device, so the positions are those that the table and the scores have room for:
  // a table much wider than its sequences costs (32 sequences of 6016 to 2048: 103 us in tables for 8192
  // positions, 190 for 65536, eight CTAs a head that each find little; 112 for 262144, long_kernel).
  const int sms = device_sms() > 0 ? device_sms() : 152;
  int ranks = 1;
  while (ranks < kMaxRanks && (S.cap > kShareThreads * 20ll * ranks ||
                               (2ll * B * S.heads * ranks <= 2ll * sms && S.cap >= 4096ll * ranks)))
    ranks *= 2;
  if (S.cap > kShareThreads * 40ll * ranks) return launch_kernel(long_kernel, dim3(unsigned(S.heads), unsigned(B)), kSelectThreads, 0, s, S);
  const auto kernel = S.cap <= kShareThreads * 20ll * ranks ? select_kernel<20> : select_kernel<40>;
  if (ranks == 1) return launch_kernel(kernel, dim3(unsigned(S.heads), unsigned(B)), kShareThreads, 0, s, S, ranks);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(ranks);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(S.heads * ranks), unsigned(B));
  cfg.blockDim = dim3(kShareThreads);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return settled(cudaLaunchKernelEx(&cfg, kernel, S, ranks));
}

cudaError_t launch_move(MoveParams& P, int B, cudaStream_t s) {
  // A list of more than a CTA's batch is shared by a cluster while there is about one CTA for each
  // SM (figures in launch_select).
  const int sms = device_sms() > 0 ? device_sms() : 152, warps = (P.width + 31) / 32;
  const int threads = warps < kMoveThreads / 32 ? 32 * warps : kMoveThreads;
  P.ranks = 1;
  while (P.ranks < kMaxRanks && 2ll * B * P.c.heads * P.ranks < sms && P.width > kMoveThreads * P.ranks) P.ranks *= 2;
  P.by_page = fast_div(uint32_t(P.c.page));
  const int cols = P.c.dim / 8;
  const auto kernel = cols <= 1   ? move_kernel<1>
                      : cols <= 2 ? move_kernel<2>
                      : cols <= 4 ? move_kernel<4>
                      : cols <= 8 ? move_kernel<8>
                                  : move_kernel<16>;
  // values that are the keys themselves move once
  const unsigned layers = P.c.k == P.c.v ? 1 : 2;
  P.scored = P.scores ? int(layers) : -1;
  const dim3 grid(unsigned(P.c.heads * P.ranks), unsigned(B), layers + (P.scores ? 1 : 0));
  if (P.ranks == 1) return launch_kernel(kernel, grid, dim3(unsigned(threads)), 0, s, P);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(P.ranks);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return settled(cudaLaunchKernelEx(&cfg, kernel, static_cast<const MoveParams&>(P)));
}

// One memory for keys and values is one set of rows.
bool same_or_apart(const dart_cache_t& c) {
  return c.k != c.v || (c.k_page_stride == c.v_page_stride && c.k_row_stride == c.v_row_stride && c.k_head_stride == c.v_head_stride);
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

namespace dart {
namespace {

int keep(const dart_cache_t* cache, const int32_t* lengths, const int32_t* path, int64_t path_stride,
         const int32_t* counts, int B, int width, const int32_t* starts, float* scores, int64_t scores_seq_stride,
         int64_t scores_head_stride, int scores_width, int32_t* out_lengths, uint32_t* device_err, void* stream) {
  if (B < 0 || B > 65535 || width < 1 || width > (1 << 30)) return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (path_stride < 0 || (B > 1 && path_stride < width) || !same_or_apart(*cache)) return DART_ERR_INVALID_ARG;
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
  P.scores = scores; P.s_seq = scores_seq_stride; P.s_head = scores_head_stride; P.s_width = scores_width;
  P.starts = starts;
  P.err = device_err;
  return launch_move(P, B, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}

bool scores_fit(const dart_cache_t& c, int B, int64_t seq_stride, int64_t head_stride, int width) {
  return width >= 0 && seq_stride >= 0 && head_stride >= 0 && (c.heads <= 1 || head_stride >= width) &&
         (B <= 1 || seq_stride >= width);
}

}  // namespace
}  // namespace dart

extern "C" int dart_kv_keep(const dart_cache_t* cache, const int32_t* lengths, const int32_t* path, int64_t path_stride,
                            const int32_t* counts, int B, int width, int32_t* out_lengths, uint32_t* device_err,
                            void* stream) {
  return dart::keep(cache, lengths, path, path_stride, counts, B, width, nullptr, nullptr, 0, 0, 0, out_lengths,
                    device_err, stream);
}

extern "C" int dart_kv_keep_scored(const dart_cache_t* cache, const int32_t* lengths, const int32_t* path,
                                   int64_t path_stride, const int32_t* counts, int B, int width, const int32_t* starts,
                                   float* scores, int64_t scores_seq_stride, int64_t scores_head_stride,
                                   int scores_width, int32_t* out_lengths, uint32_t* device_err, void* stream) {
  using namespace dart;
  if (cache && !scores_fit(*cache, B, scores_seq_stride, scores_head_stride, scores_width)) return DART_ERR_INVALID_ARG;
  if (B > 0 && (!starts || !scores)) return DART_ERR_INVALID_ARG;
  return keep(cache, lengths, path, path_stride, counts, B, width, starts, scores, scores_seq_stride,
              scores_head_stride, scores_width, out_lengths, device_err, stream);
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
  if (!scores_fit(*cache, B, scores_seq_stride, scores_head_stride, scores_width) || !same_or_apart(*cache))
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
  if (launch_select(S, B, s) != cudaSuccess) return DART_ERR_CUDA;
  MoveParams P;
  P.c = *cache;
  P.lengths = lengths;
  P.index = out_index; P.index_seq = (long long)cache->heads * keep; P.index_head = keep;
  P.counts = nullptr;
  P.out_lengths = out_lengths;
  P.width = keep; P.relative = 0;
  P.cap = int(S.cap);
  P.scores = nullptr;
  P.err = device_err;
  return launch_move(P, B, s) == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
