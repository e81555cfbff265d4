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
//   warps 8, 10  copy K tiles by TMA into a ring of swizzled stages, in turn
//   warp 9       issues the tcgen05 products, one row block after the other
//   warps 11, 12 copy the row blocks of Q (two buffers; a sequence with one or two
//                blocks keeps them there for all of its tiles)
//   warps 0-3, 4-7  add up the exponentials, each half of a block's rows
// Blocks are 64 rows where sequences have few (then the ring takes the memory:
// decoding is bound by the copy of K), else 256.
#include <cmath>
#include <type_traits>

#include "dart_tiles.cuh"

namespace dart {
namespace {

constexpr int kSumWarps = 8;
constexpr int kThreads = 13 * 32;
constexpr int kCtas = 152;
constexpr int kTile = 128;                           // positions of a tile
constexpr int kTileBytes = kTile * kColBytes;        // 64 columns of them
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxBlock = 256, kMinBlock = 64;       // rows of a block
constexpr int kMaxStages = 12, kMaxSums = 8;
constexpr int kSumThreads = kSumWarps * 32;

struct WeightParams {
  const void* q;
  const float* lse;
  float* scores;
  long long q_ts, q_hs, s_seq, s_head;
  int Hq, Hkv, G, D, T, B, N, MW;
  FastDiv by_group, by_page;
  const int32_t* lengths;
  const int32_t* starts;
  const uint32_t* mask;
  float c;
  const int32_t* table;
  long long table_stride;
  long long cap;                   // positions that a sequence's pages and scores can hold
  int page, pages, box;
  int k_slot[3];
  int block, stages, sums;         // rows of a block, K stages, S buffers (512 / block)
  uint32_t* err;
  long long wait_limit;
};

struct Shared {
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[kMaxSums], s_empty[kMaxSums];
  uint64_t drain;
  long long total, lo, hi, base;   // this CTA's share of the list, and the first unit of sequence `first`
  long long scan[kThreads / 32];
  alignas(16) float minus_l[2][kMaxBlock];   // -L of the rows in either Q buffer, -inf for a row that adds nothing
  float part[kTile];               // the second half's sums
  uint4 see[kMaxBlock];            // what each row sees of a tile
  uint32_t tmem;
  int first;
  int dead;
};

struct Seq {
  int start, n, len, lead, S, rows, blocks, tiles;
};
__device__ __forceinline__ Seq load_seq(const WeightParams& P, int b) {
  Seq c;
  const int s0 = P.starts[b], s1 = min(P.starts[b + 1], P.T);
  c.start = s0;
  c.n = s0 >= 0 && s1 > s0 ? s1 - s0 : 0;
  c.len = int(min((long long)max(P.lengths[b], 0), P.cap));
  c.S = int(min((long long)c.len + c.n, P.cap));
  c.lead = max(c.n - P.N, 0);
  c.rows = c.n * P.G;
  c.blocks = int((unsigned(c.rows) + unsigned(P.block) - 1) / unsigned(P.block));
  c.tiles = c.blocks > 0 ? (c.S + kTile - 1) / kTile : 0;
  return c;
}
__device__ __forceinline__ long long seq_cost(const WeightParams& P, const Seq& c) {
  return (long long)P.Hkv * c.tiles * c.blocks;
}
// Positions that some row of block j sees end here.
__device__ __forceinline__ int block_end(const WeightParams& P, const Seq& c, int j) {
  const int r1 = min(c.rows - j * P.block, P.block) + j * P.block;
  const int last = P.by_group.div(r1 - 1);
  return last >= c.lead ? c.S : min(c.len + last + 1, c.S);
}

// x * c / n for c <= n <= kCtas.
__device__ __forceinline__ long long share(long long x, int c, int n) {
  return x / n * c + x % n * c / n;
}

// All threads: the cost of all sequences, this CTA's share, the sequence it begins in.
__device__ void find_share(const WeightParams& P, Shared* sh) {
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
struct Tour {
  long long lin, base, hi;
  int b, h, t0, t1;
  Seq c;
  __device__ __forceinline__ bool begin(const WeightParams& P, const Shared* sh) {
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
  __device__ __forceinline__ bool resident() const { return c.blocks <= 2; }
  // Whether block j is taken for tile t: causal blocks that see nothing of it are left out,
  // unless the blocks stay in their buffers.
  __device__ __forceinline__ bool uses(const WeightParams& P, int t, int j) const {
    return resident() || block_end(P, c, j) > t * kTile;
  }
};

__device__ __forceinline__ void sum_barrier() { asm volatile("bar.sync 1, %0;" :: "n"(kSumThreads) : "memory"); }

template <typename T, int DH>
__global__ void __launch_bounds__(kThreads, 1)
weights_kernel(const WeightParams P, const __grid_constant__ CUtensorMap kmap) {
  constexpr int kStageBytes = DH * kTileBytes;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int q_half = P.block * kColBytes, q_bytes = DH * q_half;
  unsigned char* sq = smem;                              // two buffers of P.block rows
  unsigned char* ring = smem + 2 * q_bytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + P.stages * kStageBytes);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < P.stages; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], 2);                      // warps 11, 12
      mbar_init(&sh->q_empty[i], 1 + kSumWarps);         // the products, and those who read -L
    }
    for (int i = 0; i < P.sums; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->s_empty[i], kSumWarps);
    }
    mbar_init(&sh->drain, 1);
    fence_mbar_init();
    sh->dead = 0;
    sh->first = 0;
    sh->base = 0;
  }
  if (warp == 9) {
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
  Tour w;
  bool ok = true;

  if (warp == 8 || warp == 10) {
    // -------------------------------------------------------------- K tiles
    const uint32_t pid = warp == 8 ? 0u : 1u;
    uint32_t idx = 0;
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      const int32_t* table = P.table + (long long)w.b * P.table_stride;
      for (int t = w.t0; t < w.t1 && ok; ++t, ++idx) {
        if ((idx & 1u) != pid) continue;
        const int p0 = t * kTile, boxes = (min(w.c.S - p0, kTile) + P.box - 1) / P.box;
        const int at = p0 + (lane / DH) * P.box;
        const bool mine = lane / DH < boxes;
        int page = 0;
        if (mine) {
          page = table[P.by_page.div(at)];
          if (page < 0 || page >= P.pages) {
            set_dev_error(P.err, DART_DEVERR_CACHE);
            page = P.pages;                  // out of the map's range: the box arrives as zeros
          }
        }
        const uint32_t stage = idx % P.stages;
        ok = wait_warp(&sh->k_empty[stage], ((idx / P.stages) & 1u) ^ 1u, sh, limit);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&sh->k_full[stage], uint32_t(boxes * DH * P.box * kColBytes));
        __syncwarp();
        if (mine) {
          const int half = lane % DH, row = at - P.by_page.div(at) * P.page;
          auto pick = [&](int i) { return P.k_slot[i] == 0 ? w.h : P.k_slot[i] == 1 ? row : page; };
          tma_box(ring + stage * kStageBytes + half * kTileBytes + (lane / DH) * P.box * kColBytes, &kmap, 64 * half,
                  pick(0), pick(1), pick(2), &sh->k_full[stage]);
        }
      }
    }
    // no copy may land after the CTA has left: the last load of each stage is waited for
    for (uint32_t i = idx > uint32_t(P.stages) ? idx - P.stages : 0; i < idx; ++i)
      if ((i & 1u) == pid) mbar_wait_bounded(&sh->k_full[i % P.stages], (i / P.stages) & 1u, kDrainLimit);
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- tensor unit
    constexpr uint32_t type = kTypeCode<T>;
    const uint32_t id0 = (1u << 4) | (type << 7) | (type << 10) | (uint32_t(kTile >> 4) << 24);
    const uint64_t q_desc = smem_desc(smem_u32(sq), 16), k_desc = smem_desc(smem_u32(ring), 16);
    const int k_steps = (P.D + 15) / 16;
    uint32_t k_idx = 0, use = 0, load = 0;       // tiles, products and Q loads so far
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      const bool stay = w.resident();
      for (int t = w.t0; t < w.t1 && ok; ++t, ++k_idx) {
        const uint32_t stage = k_idx % P.stages;
        if (!(ok = wait_warp(&sh->k_full[stage], (k_idx / P.stages) & 1u, sh, limit))) break;
        for (int j = 0; j < w.c.blocks; ++j) {
          if (!w.uses(P, t, j)) continue;
          const uint32_t at = stay ? load + j : load;         // the Q load that this block came with
          if (!stay || t == w.t0) ok = wait_warp(&sh->q_full[at & 1u], (at >> 1) & 1u, sh, limit);
          const uint32_t s = use % P.sums;
          ok = ok && wait_warp(&sh->s_empty[s], ((use / P.sums) & 1u) ^ 1u, sh, limit);
          if (!ok) break;
          tc_after();
          const int rows = min(w.c.rows - j * P.block, P.block);
          const uint32_t id = id0 | (uint32_t((rows + 15) / 16 * 2) << 17);
          if (elect()) {
            const uint64_t kd = k_desc + uint64_t(stage * (kStageBytes >> 4));
            const uint64_t qd = q_desc + uint64_t((at & 1u) * (q_bytes >> 4));
#pragma unroll
            for (int k = 0; k < 4 * DH; ++k)
              if (k < k_steps)
                mma_ss(tmem + s * P.block, kd + (((k >> 2) * kTileBytes + (k & 3) * 32) >> 4),
                       qd + (((k >> 2) * q_half + (k & 3) * 32) >> 4), id, k > 0);
            tc_commit(&sh->s_full[s]);
            if (!stay || t == w.t1 - 1) tc_commit(&sh->q_empty[at & 1u]);
          }
          __syncwarp();
          ++use;
          if (!stay) ++load;
        }
        if (ok && elect()) tc_commit(&sh->k_empty[stage]);
        __syncwarp();
      }
      if (stay) load += w.c.blocks;
    }
    // every product has ended before the tensor memory is given back
    if (elect()) tc_commit(&sh->drain);
    mbar_wait_bounded(&sh->drain, 0, kDrainLimit);
    __syncwarp();
  } else if (warp >= 11) {
    // ------------------------------------------------------------ row blocks
    constexpr int kChunks = 8 * DH, kPer = 32 / kChunks;      // 16-byte chunks a row, rows a step
    const int chunk = lane % kChunks, sub = lane / kChunks;
    const bool inside = 8 * chunk < P.D;
    uint32_t load = 0;
    auto bring = [&](int j) {
      const uint32_t buf = load & 1u;
      ok = wait_warp(&sh->q_empty[buf], ((load >> 1) & 1u) ^ 1u, sh, limit);
      if (!ok) return;
      const int rows = min(w.c.rows - j * P.block, P.block), padded = (rows + 15) / 16 * 16;
      const T* src = static_cast<const T*>(P.q) + (inside ? 8 * chunk : 0);
      unsigned char* dst = sq + buf * q_bytes + (chunk >> 3) * q_half;
      // groups of 32 rows in turn; lane r finds row r's place and sum for all
      for (int r0 = (warp - 11) * 32; r0 < padded; r0 += 64) {
        const int g = j * P.block + min(r0 + lane, rows - 1);
        const int token = P.by_group.div(g), head = w.h * P.G + g - token * P.G;
        const long long at = (long long)(w.c.start + token) * P.q_ts + (long long)head * P.q_hs;
        float l = P.lse[(long long)(w.c.start + token) * P.Hq + head];
        const bool adds = r0 + lane < rows && fabsf(l) < INFINITY;
        if (r0 + lane < padded) sh->minus_l[buf][r0 + lane] = adds ? -l * 1.44269504088896341f : -INFINITY;
        const uint32_t on = __ballot_sync(kFull, adds);
#pragma unroll 4
        for (int u = 0; u < 32 / kPer; ++u) {
          const int r = u * kPer + sub;
          const long long from = __shfl_sync(kFull, at, r);
          // a row that adds nothing is zeros, and its exponent 0 - inf
          if (r0 + r < padded)
            cp_async16_or_zero(dst + (r0 + r) * kColBytes + (((chunk & 7) ^ (r & 7)) << 4), src + from,
                               inside && ((on >> r) & 1u));
        }
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_full[buf]);
      ++load;
    };
    for (bool more = w.begin(P, sh); more && ok; more = w.next(P)) {
      if (w.resident()) {
        for (int j = 0; j < w.c.blocks && ok; ++j) bring(j);
      } else {
        for (int t = w.t0; t < w.t1 && ok; ++t)
          for (int j = 0; j < w.c.blocks && ok; ++j)
            if (w.uses(P, t, j)) bring(j);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------------ sums
    // The schedule alone decides which barriers of the two halves are met, so a wait
    // that ran out cannot leave a warp behind: ok only turns the work off.
    const int half = warp >> 2, mine = (warp & 3) * 32 + lane;      // lane of tensor memory: the position
    const uint32_t lane_base = uint32_t(warp & 3) << 21;
    uint32_t use = 0, load = 0;
    const uint64_t c2 = pair(P.c, P.c);
    for (bool more = w.begin(P, sh); more; more = w.next(P)) {
      const bool stay = w.resident();
      float* row = P.scores + w.b * P.s_seq + w.h * P.s_head;
      const int tree = w.c.len + w.c.lead;
      const bool both = w.c.rows > 32;             // the second half has rows in some block
      for (int t = w.t0; t < w.t1; ++t) {
        const int p0 = t * kTile, p = p0 + mine, end = min(p0 + kTile, w.c.S);
        float old = 0.f;
        if (half == 0 && p < w.c.S) old = row[p];
        uint64_t sum = 0ull;
        for (int j = 0; j < w.c.blocks; ++j) {
          if (!w.uses(P, t, j)) continue;
          const uint32_t at = stay ? load + j : load, buf = at & 1u;
          const int rows = min(w.c.rows - j * P.block, P.block), cols = (rows + 15) / 16 * 16;
          const int first = P.by_group.div(j * P.block);
          // some row of the block does not see some position of the tile
          const bool masked = min(w.c.len + min(first + 1, w.c.lead), w.c.S) < end;
          if (masked) {
            sum_barrier();                         // the words of the masked block before have been read
            if (tid < P.block) {
              uint4 see = make_uint4(0, 0, 0, 0);
              if (tid < rows) {
                const int token = P.by_group.div(j * P.block + tid);
                const int plain = min(w.c.len + min(token + 1, w.c.lead), w.c.S);
                const int nodes = token >= w.c.lead ? min(min(P.N, w.c.n - w.c.lead), w.c.S - tree) : 0;
                const uint32_t* bits = P.mask + ((long long)w.b * P.N + (token - w.c.lead)) * P.MW;
                uint32_t word[5], out[4];
                const int at0 = p0 - tree, wd0 = at0 >> 5;
#pragma unroll
                for (int i = 0; i < 5; ++i) word[i] = wd0 + i >= 0 && 32 * (wd0 + i) < nodes ? bits[wd0 + i] : 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int below = max(0, min(plain - p0 - 32 * i, 32)), left = max(0, min(nodes - at0 - 32 * i, 32));
                  const uint32_t x = __funnelshift_r(word[i], word[i + 1], at0 & 31);
                  out[i] = (below >= 32 ? kFull : (1u << below) - 1u) | (x & (left >= 32 ? kFull : (1u << left) - 1u));
                }
                see = make_uint4(out[0], out[1], out[2], out[3]);
              }
              sh->see[tid] = see;
            }
            sum_barrier();
          }
          // the first half's columns and the second's, in steps of 16
          const int cut = cols <= 32 ? cols : (cols / 2 + 15) / 16 * 16;
          const int c0 = half == 0 ? 0 : cut, c1 = half == 0 ? cut : cols;
          const uint32_t s = use % P.sums;
          if (!stay || t == w.t0) ok = ok && wait_warp(&sh->q_full[buf], (at >> 1) & 1u, sh, limit);   // -L is there
          ok = ok && wait_warp(&sh->s_full[s], (use / P.sums) & 1u, sh, limit);
          if (ok) {
            tc_after();
            const uint32_t from = tmem + lane_base + s * P.block;
            const float* l = sh->minus_l[buf];
            const uint32_t* words = reinterpret_cast<const uint32_t*>(sh->see) + (warp & 3);
            auto add_up = [&](auto by_bits, auto careful) {
              uint64_t part[2] = {0ull, 0ull};
              auto add = [&](const float* x, int col) {
                const ulonglong2* l4 = reinterpret_cast<const ulonglong2*>(l + col);
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const uint64_t lk = (k & 2) ? l4[k >> 2].y : l4[k >> 2].x;
                  const uint64_t y = fma2(pair(x[k], x[k + 1]), c2, lk);
                  float a = ex2_approx(low(y)), b = ex2_approx(high(y));
                  if (decltype(by_bits)::value) {
                    a = (words[4 * (col + k)] >> lane) & 1u ? a : 0.f;
                    b = (words[4 * (col + k) + 4] >> lane) & 1u ? b : 0.f;
                  }
                  if (decltype(careful)::value) {
                    a = low(lk) == -INFINITY ? 0.f : a;
                    b = high(lk) == -INFINITY ? 0.f : b;
                  }
                  part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], pair(a, b));
                }
              };
              for (int col = c0; col < c1; col += 32) {
                float x[32];
                tmem_ld16(from + col, x);
                const bool two = col + 16 < c1;
                if (two) tmem_ld16(from + col + 16, x + 16);
                loaded<16>(x);
                add(x, col);
                if (two) {
                  loaded<16>(x + 16);
                  add(x + 16, col + 16);
                }
              }
              return add2(part[0], part[1]);
            };
            uint64_t part = masked ? add_up(std::true_type{}, std::false_type{}) : add_up(std::false_type{}, std::false_type{});
            // A row that adds nothing is zeros, and 0 * inf is NaN: where that may have
            // happened the block is added up again without those rows.
            const float both_halves = low(part) + high(part);
            if (__any_sync(kFull, both_halves != both_halves))
              part = masked ? add_up(std::true_type{}, std::true_type{}) : add_up(std::false_type{}, std::true_type{});
            sum = add2(sum, part);
            tc_before();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh->s_empty[s]);
            if (!stay || t == w.t1 - 1) mbar_arrive(&sh->q_empty[buf]);
          }
          ++use;
          if (!stay) ++load;
        }
        float gathered = low(sum) + high(sum);
        if (both) {
          if (half == 1) sh->part[mine] = gathered;
          sum_barrier();
          if (half == 0) gathered += sh->part[mine];
          sum_barrier();                           // read before the next tile's are written
        }
        if (half == 0 && p < w.c.S && ok) row[p] = old + gathered;
      }
      if (stay) load += w.c.blocks;
    }
  }

  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols));
    if (lane == 0 && sh->dead) set_dev_error(P.err, DART_DEVERR_WAIT_TIMEOUT);
  }
}

template <typename T, int DH>
cudaError_t launch(WeightParams& P, const CUtensorMap& km, cudaStream_t s) {
  constexpr int kStageBytes = DH * kTileBytes;
  const int room = 227 * 1024 - int(sizeof(Shared)) - 2 * P.block * DH * kColBytes;
  P.stages = room / kStageBytes < kMaxStages ? room / kStageBytes : kMaxStages;
  P.sums = int(kTmemCols) / P.block;
  const int smem = 2 * P.block * DH * kColBytes + P.stages * kStageBytes + int(sizeof(Shared));
  const cudaError_t e =
      settled(cudaFuncSetAttribute(weights_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (e != cudaSuccess) return e;
  const int sms = device_sms(), ctas = sms > 0 && sms < kCtas ? sms : kCtas;
  return launch_kernel(weights_kernel<T, DH>, ctas, kThreads, smem, s, P, km);
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
  P.by_group = fast_div(uint32_t(P.G));
  P.by_page = fast_div(uint32_t(c.page));
  P.lengths = lengths; P.starts = starts; P.mask = mask;
  P.c = scale * 1.44269504088896341f;
  P.table = c.table; P.table_stride = c.table_stride;
  P.cap = (long long)c.table_width * c.page;
  if (P.cap > scores_width) P.cap = scores_width;
  P.page = c.page; P.pages = c.pages; P.box = gcd(c.page, kTile);
  // few rows a sequence on average: small blocks, and the ring takes the memory
  P.block = (long long)T * P.G <= (long long)kMinBlock * B ? kMinBlock : kMaxBlock;
  P.err = device_err;
  P.wait_limit = rows_wait_limit();
  CUtensorMap km;
  if (!cache_map(c, c.k, c.k_page_stride, c.k_row_stride, c.k_head_stride, P.box, &km, P.k_slot))
    return DART_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c.dtype == DART_F16)
    e = c.dim <= 64 ? launch<__half, 1>(P, km, s) : launch<__half, 2>(P, km, s);
  else
    e = c.dim <= 64 ? launch<__nv_bfloat16, 1>(P, km, s) : launch<__nv_bfloat16, 2>(P, km, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
