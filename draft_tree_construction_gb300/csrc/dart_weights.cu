// dart_weights.cu -- K11: the attention weights that each cached position gets
// from a chunk's rows, added to what it has gathered before.
//
// Mathematics.  For position p of key head h and the rows r of its query group
// that see p (a row = a token and one of the group's queries),
//   scores[p] += sum_r 2^(c q_r . k_p - L_r),   c = scale log2 e, L_r = lse_r log2 e.
// The rows' sums are known (the attention returned them), so nothing has to be
// joined: the product is taken the other way round, S^T = K Q^T, with 128 positions
// as the tensor unit's M and a block of rows as its N.  A position is then a lane of
// tensor memory, a thread, and its sum over all rows stays in that thread's
// registers; each score is read and written once, always in the same order.
//
// One persistent CTA per SM (at most 152) takes an equal share of the list of
// (sequence, key head, tile of 128 positions), a tile costing as many row blocks
// as its sequence has.  Within a CTA:
//   12 or 16 warps  add up the exponentials: three or four groups of four warps with S buffers
//                 of their own, each every third (fourth) tile (a tile's chain from the product to
//                 the stored score is longer than the copy of a tile, and groups that
//                 share one wait for each other at every block)
//   one warp      copies K tiles by TMA into a ring of swizzled stages
//   two warps     issue the tcgen05 products, one row block after the other, each of every other
//                 group: an issue waits for the tensor unit, so that one warp's barriers would pass
//                 while nothing is computed
//   one warp      copies the row blocks of Q by TMA, a box per 64 columns (a sequence
//                 whose blocks fit in the buffers keeps them there for all of its tiles)
// Three or four tiles, a wave, are taken together: first each one's product with the first
// block, then each one's with the second, so that the groups are all fed and a block
// that does not stay is copied once for all of them.
// Blocks are whole tokens, as many as make an average sequence's blocks equal, 160 rows
// at most (128 with four groups), for which each group has an S buffer (or as many of a
// token's queries where a key head has more); what the buffers of Q leave of the shared
// memory goes to the ring (decoding is bound by the copy of K).
// -L of a block's rows lies in slots of its own, so that the next head's queries are copied
// as soon as this head's products have ended, while its last tiles are added up.
//
// Measured (GB300, bf16, 32 + 8 heads of 128, graph-replayed):
//   1 token over 4098 positions                 12.6 us: the share, the first tile and block, one chain
//   64 x 1 token over 4100..8200 positions      135..138 us, 6.0 TB/s: the keys, once
//   64 trees of 79 rows over ~1600 positions    102 us (floor 39): 85 without the masked tiles, 68 without
//     the exponentials
//   32 trees of 497 rows over ~3100 positions   517 us (floor 210)
//   2 x 2048 rows over 32768 positions          780 us, 1.24 PFLOP/s
// What bounds the last three: adding up.  With three groups it takes one 3050 cycles for 160 rows of a
// tile where the exponential unit alone would need 1920 for all three, and the next product comes 800
// later; a fourth group and the second warp of products brought 925 us down to 780.
// Tried: waves of two tiles with the groups in rotation (117 us on the trees for 106 then), a group
// for each block of a tile, the sums handed on (114 for 106), four S buffers of 128 rows that three
// groups share (118 for 103: with one warp of products a block cost much the same for any rows), all
// groups on every block, each a third of its rows (166), lanes with four positions and a quarter of the
// columns, which read a quarter of -L (112 for 103), one thread for all products (108 for 103).
#include <cmath>
#include <type_traits>

#include "dart_tiles.cuh"

namespace dart {
namespace {

// By groups: the threads of a CTA, and the rows of a block, an S buffer for each group.
__host__ __device__ constexpr int threads_of(int groups) { return (4 * groups + 4) * 32; }
__host__ __device__ constexpr int rows_of(int groups) { return groups == 3 ? 160 : 128; }
constexpr int kCtas = 152;
constexpr int kTile = 128;                           // positions of a tile
constexpr int kTileBytes = kTile * kColBytes;        // 64 columns of them
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12, kMaxSums = 4, kMaxQ = 4, kSlots = 8;

struct WeightParams {
  const void* q;
  const float* lse;
  float* scores;
  long long q_ts, q_hs, s_seq, s_head;
  int Hq, Hkv, G, D, T, B, N, MW;
  FastDiv by_page;
  const int32_t* lengths;
  const int32_t* starts;
  const uint32_t* mask;
  float c;
  const int32_t* table;
  long long table_stride;
  long long cap;                   // positions that a sequence's pages and scores can hold
  int page, pages, box;
  int k_slot[3];
  int tokens, queries_of;          // of a block: its tokens, the queries of each
  int parts;                       // blocks that a token takes (more than one only with one token a block)
  FastDiv by_part, by_queries;
  int block, columns;              // rows of a buffer, tensor memory columns from one S buffer to the next
  int stages, sums, queries;       // K stages, S buffers of a group, Q buffers
  uint32_t* err;
  long long wait_limit;
};

template <int G>
struct Shared {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t q_full[kMaxQ], q_empty[kMaxQ];
  uint64_t l_full[kSlots], l_empty[kSlots];
  uint64_t s_full[G * kMaxSums], s_empty[G * kMaxSums];
  uint64_t drain;
  long long total, lo, hi, base;   // this CTA's share of the list, and the first unit of sequence `first`
  long long scan[threads_of(G) / 32];
  alignas(16) float minus_l[kSlots][rows_of(G)];  // -L of the rows of a block, -inf for a row that adds nothing
  alignas(16) uint32_t see[G][4][rows_of(G)];   // what each row sees of a group's tile, 32 positions a word
  uint32_t tmem;
  int first;
  int dead;
};

struct Seq {
  int start, n, len, lead, S, blocks, tiles;
};
__device__ __forceinline__ Seq load_seq(const WeightParams& P, int b) {
  Seq c;
  const int s0 = P.starts[b], s1 = min(P.starts[b + 1], P.T);
  c.start = s0;
  c.n = s0 >= 0 && s1 > s0 ? s1 - s0 : 0;
  c.len = int(min((long long)max(P.lengths[b], 0), P.cap));
  c.S = int(min((long long)c.len + c.n, P.cap));
  c.lead = max(c.n - P.N, 0);
  c.blocks = P.parts > 1 ? c.n * P.parts : (c.n + P.tokens - 1) / P.tokens;
  c.tiles = c.blocks > 0 ? (c.S + kTile - 1) / kTile : 0;
  return c;
}
__device__ __forceinline__ long long seq_cost(const WeightParams& P, const Seq& c) {
  return (long long)P.Hkv * c.tiles * c.blocks;
}
// A block of rows: row r is query q0 + r % queries of token t0 + r / queries.
struct Block {
  int t0, q0, tokens, queries, rows;
};
__device__ __forceinline__ Block block_of(const WeightParams& P, const Seq& c, int j) {
  Block k;
  if (P.parts == 1) {
    k.t0 = j * P.tokens;
    k.q0 = 0;
    k.tokens = min(P.tokens, c.n - k.t0);
    k.queries = P.G;
  } else {
    k.t0 = P.by_part.div(j);
    k.q0 = (j - k.t0 * P.parts) * P.queries_of;
    k.tokens = 1;
    k.queries = min(P.queries_of, P.G - k.q0);
  }
  k.rows = k.tokens * k.queries;
  return k;
}
// The first block of which some row sees positions from p on (p < S): they all do from there.
__device__ __forceinline__ int first_block(const WeightParams& P, const Seq& c, int p) {
  const int token = min(max(p - c.len, 0), c.lead);       // sees p, and so do those behind it
  return P.parts > 1 ? token * P.parts : token / P.tokens;
}

// x * c / n for c <= n <= kCtas.
__device__ __forceinline__ long long share(long long x, int c, int n) {
  return x / n * c + x % n * c / n;
}

// All threads: the cost of all sequences, this CTA's share, the sequence it begins in.
template <int G>
__device__ void find_share(const WeightParams& P, Shared<G>* sh) {
  constexpr int kThreads = threads_of(G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long before = 0, lo = 0;
  bool bad = false;
  for (int pass = 0; pass < 2; ++pass) {
    before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      const int b = b0 + tid;
      long long cost = 0;
      if (b < P.B) {
        const Seq c = load_seq(P, b);
        cost = seq_cost(P, c);
        bad |= P.lengths[b] < 0 || (c.n > 0 && (long long)P.lengths[b] + c.n > P.cap);
      }
      long long incl = cost;
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      __syncthreads();
      if (lane == 31) sh->scan[warp] = incl;
      __syncthreads();
      long long lower = before;
      for (int w = 0; w < kThreads / 32; ++w) {
        const long long x = sh->scan[w];
        if (w < warp) lower += x;
        before += x;
      }
      incl += lower;
      if (pass == 1 && cost > 0 && lo >= incl - cost && lo < incl) {
        sh->first = b;
        sh->base = incl - cost;
      }
    }
    if (pass == 0) {
      lo = share(before, blockIdx.x, gridDim.x);
      if (tid == 0) {
        sh->total = before;
        sh->lo = lo;
        sh->hi = share(before, blockIdx.x + 1, gridDim.x);
      }
    }
  }
  if (bad && blockIdx.x == 0) set_dev_error(P.err, DART_DEVERR_CACHE);
}

// A CTA's walk over its share, consecutive tiles of one head at a time.  A tile
// belongs to the CTA in whose share its first block lies.
template <int G>
struct Tour {
  long long lin, base, hi;
  int b, h, t0, t1;
  Seq c;
  __device__ __forceinline__ bool begin(const WeightParams& P, const Shared<G>* sh) {
    hi = sh->hi;
    if (sh->lo >= hi) return false;
    b = sh->first;
    base = sh->base;
    c = load_seq(P, b);
    lin = (sh->lo - base + c.blocks - 1) / c.blocks;
    return next(P);
  }
  __device__ __forceinline__ bool next(const WeightParams& P) {
    for (;;) {
      if (c.blocks > 0) {
        const long long all = (long long)P.Hkv * c.tiles;
        const long long end = min(all, (hi - base + c.blocks - 1) / c.blocks);
        if (lin < end) {
          h = int(lin / c.tiles);
          t0 = int(lin - (long long)h * c.tiles);
          t1 = int(min((long long)c.tiles, t0 + (end - lin)));
          lin += t1 - t0;
          return true;
        }
        base += all * c.blocks;
      }
      if (base >= hi || ++b >= P.B) return false;
      c = load_seq(P, b);
      lin = 0;
    }
  }
  __device__ __forceinline__ bool resident(const WeightParams& P) const { return c.blocks <= P.queries; }
  // The first block taken for the wave from tile t on: causal blocks that see nothing of
  // it are left out, unless the blocks stay in their buffers.
  __device__ __forceinline__ int begin_block(const WeightParams& P, int t) const {
    return resident(P) ? 0 : first_block(P, c, t * kTile);
  }
  __device__ __forceinline__ int wave(int t) const { return min(G, t1 - t); }
};

// A place in a ring of n, and the parity of its round.
struct Ring {
  uint32_t at = 0, round = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == uint32_t(n)) {
      at = 0;
      round ^= 1;
    }
  }
  __device__ __forceinline__ Ring plus(int k, int n) const {       // k <= n
    Ring r = *this;
    r.at += k;
    if (r.at >= uint32_t(n)) {
      r.at -= n;
      r.round ^= 1;
    }
    return r;
  }
};

template <int ID, int N>
__device__ __forceinline__ void named_barrier(int offset = 0) {
  asm volatile("bar.sync %0, %1;" :: "r"(ID + offset), "n"(N) : "memory");
}
// What the rows of block k see of the positions from p0 on, by a group's 128 threads.  Not
// inlined: it is rare, and the sums need the registers.
template <int G>
__device__ __noinline__ void look(const WeightParams& P, Shared<G>* sh, const Seq& c, const Block& k, int b, int group, int mine,
                                  int p0, const float* minus_l) {
  const int tree = c.len + c.lead, at0 = p0 - tree, wd0 = at0 >> 5;
  for (int r = mine; r < (k.rows + 15) / 16 * 16; r += 128) {
    const int token = k.t0 + (P.parts == 1 ? P.by_queries.div(r) : 0);
    const bool on = r < k.rows && minus_l[r] > -INFINITY;        // a row that adds nothing sees nothing
    const int plain = on ? min(c.len + min(token + 1, c.lead), c.S) : 0;
    const int nodes = on && token >= c.lead ? min(min(P.N, c.n - c.lead), c.S - tree) : 0;
    const uint32_t* bits = P.mask + ((long long)b * P.N + (token - c.lead)) * P.MW;
    uint32_t word[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) word[i] = wd0 + i >= 0 && 32 * (wd0 + i) < nodes ? bits[wd0 + i] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int below = max(0, min(plain - p0 - 32 * i, 32)), left = max(0, min(nodes - at0 - 32 * i, 32));
      const uint32_t x = __funnelshift_r(word[i], word[i + 1], at0 & 31);
      sh->see[group][i][r] = (below >= 32 ? kFull : (1u << below) - 1u) | (x & (left >= 32 ? kFull : (1u << left) - 1u));
    }
  }
}

template <typename T, int DH, int G>
__global__ void __launch_bounds__(threads_of(G), 1)
weights_kernel(const __grid_constant__ WeightParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap) {
  constexpr int kStageBytes = DH * kTileBytes, kSumWarps = 4 * G, kThreads = threads_of(G);
  extern __shared__ __align__(1024) unsigned char smem[];
  const int q_half = P.block * kColBytes, q_bytes = DH * q_half;
  unsigned char* sq = smem;                              // the buffers of Q
  unsigned char* ring = smem + P.queries * q_bytes;
  Shared<G>* sh = reinterpret_cast<Shared<G>*>(ring + P.stages * kStageBytes);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P.stages; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 2);                     // both warps of products, the one that has none of the tile too
    }
    for (int i = 0; i < P.queries; ++i) {
      mbar_init(&sh->q_full[i], 1);
      mbar_init(&sh->q_empty[i], 2);                     // both warps of products
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh->l_full[i], 1);
      mbar_init(&sh->l_empty[i], kSumWarps);
    }
    for (int i = 0; i < G * P.sums; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->s_empty[i], 4);                     // the group's warps
    }
    mbar_init(&sh->drain, 2);
    fence_mbar_init();
    sh->dead = 0;
    sh->first = 0;
    sh->base = 0;
  }
  // the rows that fill a block up to a multiple of 16 are never copied: zeros, so that they
  // give no NaN
  const int copied = P.tokens * P.queries_of;
  for (int i = tid; i < P.queries * DH * (P.block - copied) * 8; i += kThreads) {
    const int half = i / ((P.block - copied) * 8), at = i - half * (P.block - copied) * 8;
    *reinterpret_cast<uint4*>(sq + half * q_half + copied * kColBytes + at * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_async();
  if (warp == kSumWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  find_share(P, sh);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh->tmem;
  const long long limit = P.wait_limit;
  Tour<G> w;
  bool ok = true;

  if (warp == kSumWarps) {
    // -------------------------------------------------------------- K tiles
    uint32_t idx = 0;
    Ring stage;
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      const int32_t* table = P.table + (long long)w.b * P.table_stride;
      const int at = (lane / DH) * P.box;                  // this lane's box in a tile
      int next = w.t0 * kTile + at < w.c.S && at < kTile ? table[P.by_page.div(w.t0 * kTile + at)] : 0;
      for (int t = w.t0; t < w.t1 && ok; ++t, ++idx, stage.next(P.stages)) {
        const int p0 = t * kTile, boxes = (min(w.c.S - p0, kTile) + P.box - 1) / P.box;
        const bool mine = lane / DH < boxes;
        int page = next;
        // the next tile's page is on its way meanwhile
        if (t + 1 < w.t1 && at < kTile && p0 + kTile + at < w.c.S) next = table[P.by_page.div(p0 + kTile + at)];
        if (mine && (page < 0 || page >= P.pages)) {
          set_dev_error(P.err, DART_DEVERR_CACHE);
          page = P.pages;                    // out of the map's range: the box arrives as zeros
        }
        ok = wait_warp(&sh->k_empty[stage.at], stage.round ^ 1u, sh, limit);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sh->k_full[stage.at], uint32_t(boxes * DH * P.box * kColBytes));
        __syncwarp();
        if (mine) {
          const int half = lane % DH, row = p0 + at - P.by_page.div(p0 + at) * P.page;
          auto pick = [&](int i) { return P.k_slot[i] == 0 ? w.h : P.k_slot[i] == 1 ? row : page; };
          tma_box(ring + stage.at * kStageBytes + half * kTileBytes + at * kColBytes, &kmap, 64 * half,
                  pick(0), pick(1), pick(2), &sh->k_full[stage.at]);
        }
      }
    }
    // no copy may land after the CTA has left: the last load of each stage is waited for
    for (uint32_t i = idx > uint32_t(P.stages) ? idx - P.stages : 0; i < idx; ++i)
      mbar_wait_bounded(&sh->k_full[i % P.stages], (i / P.stages) & 1u, kDrainLimit);
    __syncwarp();
  } else if (warp == kSumWarps + 1 || warp == kSumWarps + 2) {
    // ---------------------------------------------------------- tensor unit
    constexpr uint32_t type = kTypeCode<T>;
    const uint32_t id0 = (1u << 4) | (type << 7) | (type << 10) | (uint32_t(kTile >> 4) << 24);
    const uint64_t q_desc = smem_desc(smem_u32(sq), 16), k_desc = smem_desc(smem_u32(ring), 16);
    const int k_steps = (P.D + 15) / 16;
    const uint64_t half = uint64_t(q_half >> 4);
    constexpr int kOwn = (G + 1) / 2;                        // this warp has every other group
    const int own = warp - kSumWarps - 1;
    Ring stage, load, s[kOwn];
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      const bool stay = w.resident(P);
      const int blocks = w.c.blocks;
      for (int t = w.t0; t < w.t1 && ok; t += G) {
        const int tiles = w.wave(t), begin = w.begin_block(P, t);
        const bool ends = t + G >= w.t1;               // the segment's last wave
        for (int j = begin; j < blocks && ok; ++j) {
          const Ring at = stay ? load.plus(j, P.queries) : load;       // the Q load that this block came with
          const int rows = P.parts == 1 && j + 1 < blocks ? P.tokens * P.G : block_of(P, w.c, j).rows;
          const uint32_t id = id0 | (uint32_t((rows + 15) / 16 * 2) << 17);
          const uint64_t qd = q_desc + uint64_t(at.at * (q_bytes >> 4));
          if (!stay || t == w.t0) ok = wait_warp(&sh->q_full[at.at], at.round, sh, limit);
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const int g = 2 * i + own;
            if (g >= tiles || !ok) break;
            const Ring k_at = stage.plus(g, P.stages);
            const uint32_t buf = uint32_t(g) * P.sums + s[i].at, d = tmem + buf * P.columns;
            const uint64_t kd = k_desc + uint64_t(k_at.at * (kStageBytes >> 4));
            if (j == begin) ok = wait_warp(&sh->k_full[k_at.at], k_at.round, sh, limit);
            ok = ok && wait_warp(&sh->s_empty[buf], s[i].round ^ 1u, sh, limit);
            if (!ok) break;
            tc_after();
            if (elect()) {
              if (k_steps == 4 * DH) {
#pragma unroll
                for (int k = 0; k < 4 * DH; ++k)
                  mma_ss(d, kd + (((k >> 2) * kTileBytes + (k & 3) * 32) >> 4), qd + (k < 4 ? 0 : half) + (((k & 3) * 32) >> 4), id, k > 0);
              } else {
                for (int k = 0; k < k_steps; ++k)
                  mma_ss(d, kd + (((k >> 2) * kTileBytes + (k & 3) * 32) >> 4), qd + (k < 4 ? 0 : half) + (((k & 3) * 32) >> 4), id, k > 0);
              }
              tc_commit(&sh->s_full[buf]);
              if (j + 1 == blocks) tc_commit(&sh->k_empty[k_at.at]);
            }
            __syncwarp();
            s[i].next(P.sums);
          }
          if (ok && (!stay || ends) && elect()) tc_commit(&sh->q_empty[at.at]);
          // this warp sees the other's tiles arrive and gives them up too: a stage's round is told by one
          // bit, so neither may miss one
          for (int g = 1 - own; j == begin && g < tiles && ok; g += 2) {
            const Ring k_at = stage.plus(g, P.stages);
            ok = wait_warp(&sh->k_full[k_at.at], k_at.round, sh, limit);
            if (ok && lane == 0) mbar_arrive(&sh->k_empty[k_at.at]);
            __syncwarp();
          }
          __syncwarp();
          if (!stay) load.next(P.queries);
        }
        stage = stage.plus(tiles, P.stages);
      }
      if (stay) load = load.plus(blocks, P.queries);
    }
    // every product has ended before the tensor memory is given back
    if (elect()) tc_commit(&sh->drain);
    mbar_wait_bounded(&sh->drain, 0, kDrainLimit);
    __syncwarp();
  } else if (warp == kSumWarps + 3) {
    // ------------------------------------------------------------ row blocks
    constexpr int kPer = rows_of(G) / 32;
    Ring load, slot;
    uint32_t loads = 0;
    auto bring = [&](int j) {
      const uint32_t buf = load.at;
      const Block k = block_of(P, w.c, j);
      // the rows' sums are on their way while the buffer is waited for
      float l[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = min(32 * i + lane, k.rows - 1);
        const int token = P.parts == 1 ? P.by_queries.div(r) : 0, q = k.q0 + r - token * k.queries;
        l[i] = 32 * i < k.rows ? P.lse[(long long)(w.c.start + k.t0 + token) * P.Hq + w.h * P.G + q] : 0.f;
      }
      ok = wait_warp(&sh->l_empty[slot.at], slot.round ^ 1u, sh, limit);
      if (!ok) return;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (32 * i + lane < P.block) {
          const bool adds = 32 * i + lane < k.rows && fabsf(l[i]) < INFINITY;
          sh->minus_l[slot.at][32 * i + lane] = adds ? -l[i] * 1.44269504088896341f : -INFINITY;
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->l_full[slot.at]);
      slot.next(kSlots);
      ok = wait_warp(&sh->q_empty[buf], load.round ^ 1u, sh, limit);
      if (!ok) return;
      // whole boxes: what lies behind the block's rows adds nothing
      if (lane == 0) mbar_expect_tx(&sh->q_full[buf], uint32_t(DH * P.tokens * P.queries_of * kColBytes));
      __syncwarp();
      if (lane < DH)
        tma_box(sq + buf * q_bytes + lane * q_half, &qmap, 64 * lane, w.h * P.G + k.q0, w.c.start + k.t0, 0, &sh->q_full[buf]);
      load.next(P.queries);
      ++loads;
    };
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      if (w.resident(P)) {
        for (int j = 0; j < w.c.blocks && ok; ++j) bring(j);
      } else {
        for (int t = w.t0; t < w.t1 && ok; t += G)
          for (int j = w.begin_block(P, t); j < w.c.blocks && ok; ++j) bring(j);
      }
    }
    for (uint32_t i = loads > uint32_t(P.queries) ? loads - P.queries : 0; i < loads; ++i)
      mbar_wait_bounded(&sh->q_full[i % P.queries], (i / P.queries) & 1u, kDrainLimit);
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ sums
    // The schedule alone decides which barriers a group's warps meet at, so a wait that
    // ran out cannot leave a warp behind: ok only turns the work off.
    const int group = warp >> 2, mine = (warp & 3) * 32 + lane;     // lane of tensor memory: the position
    const uint32_t lane_base = uint32_t(warp & 3) << 21;
    Ring s, load;
    const uint64_t c2 = pair(P.c, P.c);
    for (bool more = w.begin(P, sh); more; more = w.next(P)) {
      const bool stay = w.resident(P);
      float* row = P.scores + w.b * P.s_seq + w.h * P.s_head;
      for (int t = w.t0; t < w.t1; t += G) {
        // all groups see every block's rows arrive, so that none gives them up before their time
        const bool here = group < w.wave(t);
        const int p0 = (t + group) * kTile, p = p0 + mine, end = min(p0 + kTile, w.c.S);
        const bool writes = here && p < w.c.S;
        float old = 0.f;
        if (writes) old = row[p];
        uint64_t sum = 0ull;
        for (int j = w.begin_block(P, t); j < w.c.blocks; ++j) {
          const Ring at = stay ? load.plus(j, kSlots) : load;
          if (!stay || t == w.t0) ok = ok && wait_warp(&sh->l_full[at.at], at.round, sh, limit);
          if (!stay) load.next(kSlots);
          if (!here) {
            if (!stay && lane == 0) mbar_arrive(&sh->l_empty[at.at]);
            continue;
          }
          const Block k = block_of(P, w.c, j);
          const int cols = (k.rows + 15) / 16 * 16;
          // some row of the block does not see some position of the tile
          const bool masked = min(w.c.len + min(k.t0 + 1, w.c.lead), w.c.S) < end;
          if (masked) {
            named_barrier<1, 128>(group);          // the words of the masked block before have been read
            look(P, sh, w.c, k, w.b, group, mine, p0, sh->minus_l[at.at]);
            named_barrier<1, 128>(group);
          }
          const uint32_t buf = uint32_t(group) * P.sums + s.at;
          ok = ok && wait_warp(&sh->s_full[buf], s.round, sh, limit);
          if (ok) {
            tc_after();
            const uint32_t from = tmem + lane_base + buf * P.columns;
            const float* l = sh->minus_l[at.at];
            const uint32_t* words = sh->see[group][warp & 3];
            uint64_t part[2] = {0ull, 0ull};
            auto fast = [&](const float* x, int col) {
              const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(l + col);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const ulonglong2 lk = l4[k >> 2];
                const uint64_t y0 = fma2(pair(x[k], x[k + 1]), c2, lk.x), y1 = fma2(pair(x[k + 2], x[k + 3]), c2, lk.y);
                part[0] = add2(part[0], pair(ex2_approx(low(y0)), ex2_approx(high(y0))));
                part[1] = add2(part[1], pair(ex2_approx(low(y1)), ex2_approx(high(y1))));
              }
            };
            // what a row does not see is left out whatever the product is
            const uint32_t bit = 1u << lane;
            auto seen = [&](const float* x, int col) {
              const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(l + col);
              const uint4* w4 = reinterpret_cast<const uint4*>(words + col);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const ulonglong2 lk = l4[k >> 2];
                const uint4 wk = w4[k >> 2];
                const uint64_t y0 = fma2(pair(x[k], x[k + 1]), c2, lk.x), y1 = fma2(pair(x[k + 2], x[k + 3]), c2, lk.y);
                const float a0 = wk.x & bit ? low(y0) : -INFINITY, a1 = wk.y & bit ? high(y0) : -INFINITY,
                            a2 = wk.z & bit ? low(y1) : -INFINITY, a3 = wk.w & bit ? high(y1) : -INFINITY;
                part[0] = add2(part[0], pair(ex2_approx(a0), ex2_approx(a1)));
                part[1] = add2(part[1], pair(ex2_approx(a2), ex2_approx(a3)));
              }
            };
            // with three groups the next columns are on their way while these are added up
            auto all = [&](auto&& add) {
              if constexpr (G < 4) {
                float x[2][16];
                tmem_ld16(from, x[0]);
                for (int col = 0; col < cols; col += 32) {
                  loaded<16>(x[0]);
                  if (col + 16 < cols) tmem_ld16(from + col + 16, x[1]);
                  add(x[0], col);
                  if (col + 16 < cols) {
                    loaded<16>(x[1]);
                    if (col + 32 < cols) tmem_ld16(from + col + 32, x[0]);
                    add(x[1], col + 16);
                  }
                }
              } else {
#pragma unroll 1
                for (int col = 0; col < cols; col += 16) {
                  float x[16];
                  tmem_ld16(from + col, x);
                  loaded<16>(x);
                  add(x, col);
                }
              }
            };
            if (masked) {
              all(seen);
            } else {
              all(fast);
              // a row that adds nothing is zeros or what lies behind the chunk, which may hold anything:
              // where that gave NaN the block is added up once more without those rows
              const uint64_t both = add2(part[0], part[1]);
              if (__any_sync(kFull, low(both) + high(both) != low(both) + high(both))) {
                part[0] = part[1] = 0ull;
#pragma unroll 1
                for (int col = 0; col < cols; col += 16) {
                  float x[16];
                  tmem_ld16(from + col, x);
                  loaded<16>(x);
#pragma unroll
                  for (int k = 0; k < 16; ++k)
                    if (l[col + k] > -INFINITY) part[0] = add2(part[0], pair(ex2_approx(fmaf(x[k], P.c, l[col + k])), 0.f));
                }
              }
            }
            sum = add2(sum, add2(part[0], part[1]));
            tc_before();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->s_empty[buf]);
            if (!stay) mbar_arrive(&sh->l_empty[at.at]);
          }
          s.next(P.sums);
        }
        if (writes && ok) row[p] = old + (low(sum) + high(sum));
      }
      if (stay) {
        __syncwarp();
        if (lane == 0)
          for (int j = 0; j < w.c.blocks; ++j) mbar_arrive(&sh->l_empty[load.plus(j, kSlots).at]);
        load = load.plus(w.c.blocks, kSlots);
      }
    }
  }

  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kSumWarps + 1) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols));
    if (lane == 0 && sh->dead) set_dev_error(P.err, DART_DEVERR_WAIT_TIMEOUT);
  }
}

// The queries as a map (columns, query, token, one) with a box of a block's queries and tokens by 64 columns.
bool query_map(const WeightParams& P, const dart_cache_t& c, CUtensorMap* map) {
  const EncodeFn encode = tensor_map_encoder();
  if (!encode) return false;
  // a dimension of one is never stepped along: any valid stride serves
  const cuuint64_t row = cuuint64_t(P.D) * 2;
  const cuuint64_t dims[4] = {cuuint64_t(P.D), cuuint64_t(P.Hq), cuuint64_t(P.T), 1};
  const cuuint64_t strides[3] = {P.Hq > 1 ? cuuint64_t(P.q_hs) * 2 : row, P.T > 1 ? cuuint64_t(P.q_ts) * 2 : row, row};
  if (strides[0] == 0 || strides[1] == 0) return false;
  const cuuint32_t boxes[4] = {64, cuuint32_t(P.queries_of), cuuint32_t(P.tokens), 1}, steps[4] = {1, 1, 1, 1};
  return encode(map, c.dtype == DART_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(P.q), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DH, int G>
cudaError_t launch(WeightParams& P, const CUtensorMap& km, const CUtensorMap& qm, cudaStream_t s) {
  constexpr int kStageBytes = DH * kTileBytes;
  // A wave's stages of K and one more at least, then buffers of Q so that the next head's
  // blocks can come while this one's are used, then stages again.
  constexpr int kMost = 227 * 1024;
  const int room = kMost - int(sizeof(Shared<G>)), q = P.block * DH * kColBytes;
  P.queries = (room - 4 * kStageBytes) / q;
  P.queries = P.queries < 2 ? 2 : P.queries > kMaxQ ? kMaxQ : P.queries;
  P.stages = (room - P.queries * q) / kStageBytes;
  P.stages = P.stages < kMaxStages ? P.stages : kMaxStages;
  P.columns = (P.block + 31) / 32 * 32;
  P.sums = int(kTmemCols) / P.columns / G;
  P.sums = P.sums < kMaxSums ? P.sums : kMaxSums;
  const int smem = P.queries * q + P.stages * kStageBytes + int(sizeof(Shared<G>));
  // the same limit from every call: it is the kernel's, not the launch's, and a call of another shape
  // in another thread may come between this line and the launch
  const cudaError_t e =
      settled(cudaFuncSetAttribute(weights_kernel<T, DH, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost));
  if (e != cudaSuccess) return e;
  const int sms = device_sms(), ctas = sms > 0 && sms < kCtas ? sms : kCtas;
  return launch_kernel(weights_kernel<T, DH, G>, ctas, threads_of(G), smem, s, P, km, qm);
}

template <typename T>
cudaError_t launch_type(WeightParams& P, int groups, const CUtensorMap& km, const CUtensorMap& qm, cudaStream_t s) {
  if (groups == 3) return P.D <= 64 ? launch<T, 1, 3>(P, km, qm, s) : launch<T, 2, 3>(P, km, qm, s);
  return P.D <= 64 ? launch<T, 1, 4>(P, km, qm, s) : launch<T, 2, 4>(P, km, qm, s);
}

}  // namespace
}  // namespace dart

extern "C" int dart_attention_weights(const void* q, int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                                      int T, int B, const int32_t* lengths, const int32_t* starts,
                                      const uint32_t* mask, int N, float scale, const dart_cache_t* cache,
                                      const float* lse, float* scores, int64_t scores_seq_stride,
                                      int64_t scores_head_stride, int scores_width, uint32_t* device_err,
                                      void* stream) {
  using namespace dart;
  if (T < 0 || T > (1 << 26) || B < 0 || q_heads < 1 || q_heads > 65535 || N < 0 || N > kMaxN || scores_width < 0)
    return DART_ERR_INVALID_ARG;
  if ((long long)T * q_heads >= (1ll << 31)) return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (q_heads % cache->heads != 0 || !std::isfinite(scale * 1.44269504f)) return DART_ERR_INVALID_ARG;
  if (scores_seq_stride < 0 || scores_head_stride < 0 || (cache->heads > 1 && scores_head_stride < scores_width) ||
      (B > 1 && scores_seq_stride < scores_width))
    return DART_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DART_OK;
  if (cache->pages < 1 || cache->table_width < 1) return DART_ERR_INVALID_ARG;
  if (!aligned16(q) || !mult8(q_token_stride, q_head_stride) || !lengths || !starts || (N > 0 && !mask) || !lse ||
      !scores)
    return DART_ERR_INVALID_ARG;
  const dart_cache_t& c = *cache;
  WeightParams P;
  P.q = q; P.lse = lse; P.scores = scores;
  P.q_ts = q_token_stride; P.q_hs = q_head_stride;
  P.s_seq = scores_seq_stride; P.s_head = scores_head_stride;
  P.Hq = q_heads; P.Hkv = c.heads; P.G = q_heads / c.heads; P.D = c.dim;
  P.T = T; P.B = B; P.N = N; P.MW = (N + 31) / 32;
  P.by_page = fast_div(uint32_t(c.page));
  P.lengths = lengths; P.starts = starts; P.mask = mask;
  P.c = scale * 1.44269504088896341f;
  P.table = c.table; P.table_stride = c.table_stride;
  P.cap = (long long)c.table_width * c.page;
  if (P.cap > scores_width) P.cap = scores_width;
  P.page = c.page; P.pages = c.pages; P.box = gcd(c.page, kTile);
  // Three groups of warps where an average sequence's rows stay in shared memory, four where they are
  // copied again for each wave (three for four: 64 trees of 79 rows 103 us for 111, 2 x 512 rows over
  // 16384 positions 124 for 108, 2 x 2048 over 32768 922 for 780).
  const long long rows = ((long long)T + B - 1) / B * (q_heads / c.heads);
  const int groups = rows <= (c.dim <= 64 ? 4 : 2) * rows_of(3) ? 3 : 4;
  // an average sequence's tokens in equal blocks
  const int most = rows_of(groups);
  P.queries_of = P.G < most ? P.G : most;
  P.parts = (P.G + P.queries_of - 1) / P.queries_of;
  const int fit = most / P.queries_of, tokens = int(((long long)T + B - 1) / B), blocks = (tokens + fit - 1) / fit;
  P.tokens = P.parts > 1 ? 1 : (tokens + blocks - 1) / blocks;
  P.block = (P.tokens * P.queries_of + 15) / 16 * 16;
  P.by_part = fast_div(uint32_t(P.parts));
  P.by_queries = fast_div(uint32_t(P.G));
  P.err = device_err;
  P.wait_limit = rows_wait_limit();
  CUtensorMap km;
  if (!cache_map(c, c.k, c.k_page_stride, c.k_row_stride, c.k_head_stride, P.box, &km, P.k_slot))
    return DART_ERR_UNSUPPORTED;
  CUtensorMap qm;
  if (!query_map(P, c, &qm)) return DART_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c.dtype == DART_F16)
    e = launch_type<__half>(P, groups, km, qm, s);
  else
    e = launch_type<__nv_bfloat16>(P, groups, km, qm, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
