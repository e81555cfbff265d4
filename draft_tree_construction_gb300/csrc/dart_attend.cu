// dart_attend.cu -- K7: attention of a chunk of new tokens over a paged cache,
// the chunk's tail being a tree with packed ancestor-or-self masks.
//
// Mathematics.  For the rows of one key head (a row = a token and one of the
// head group's queries) and tiles of 128 cache positions,
//   S = Q K^T,  m' = max(m, rowmax S),  P = 2^(c S - m'),  l' = l 2^(m - m') + rowsum P,
//   O' = O 2^(m - m') + P V,            out = O / l,       c = scale * log2 e,
// one pass over the cache, fp32 statistics, P rounded to the cache's type for
// the second product.  m only moves when the maximum has grown by more than
// 2^8 (the factor 2^(m - m') then touches O); p stays below 2^8 and l above 2^-0
// until then, which neither fp16 nor fp32 minds.
//
// One persistent CTA per SM (at most 152).  The work is the list of (sequence, key head,
// block of 256 rows, tile of 128 positions), cut into equal contiguous spans,
// so a block's tiles may be spread over several CTAs: each leaves (m, l, O) of
// its part in the workspace and the join kernel merges them in a fixed order.
// Within a CTA:
//   warps 8, 11 copy K and V tiles by TMA, one box per page and 64 columns,
//               into a ring of swizzled shared-memory stages; they take the
//               loads in turn, because a box costs its warp about 100 cycles
//   warps 9, 10 issue the tcgen05 products of one 128-row half each: S into
//               TMEM, P V into TMEM, P being read from TMEM where it replaced S.
//               One warp for both left the tensor unit idle for the 900 cycles
//               a tile that its waits and commits take (61% busy).
//   warps 0-3, 4-7   softmax of one half each, a thread per row; while one
//               half's softmax runs, the tensor unit works on the other's
//
// Measured (GB300, bf16, 32 + 8 heads of 128, both kernels):
//   64 x 1 token over 4100..8200 positions    247 us, 6.4 TB/s: the cache, once
//   2 x 2048 tokens over 32768 positions     1340 us, 1.43 PFLOP/s (fp16; 1.21 when
//     the card holds its power limit for seconds): a tile takes 3000 cycles, 2048
//     of them in the tensor unit; the chain S -> softmax (1400) -> P V -> next S
//     of a half is what is longer.  Handing P over in two halves: 1480 us.  Two
//     threads a row, 64 positions each: 1460 us (the exponentials, 512 cycles a
//     half's tile, and the row's exchange leave the softmax at 1500).
//   32 trees of 497 rows over ~3100 positions  721 us, 1.11 PFLOP/s of what is seen
//     (830 us when the card holds its power limit for seconds)
//   64 trees of 79 rows over ~1600 positions   181 us: 316 rows are a block of
//     256 and one of 60, so the cache passes through the CTAs twice (5 TB/s from
//     L2 and memory), and six block changes a CTA take a tenth.  Dealing the
//     tiles of a short block to both halves and merging them: 199 us.  Moving a
//     span's end to a block's end within 4 tiles, so that fewer blocks are joined:
//     178 us for 175.5 here, 95 for 103 in 128 trees of 256 rows over ~450
//     positions, 8.6 for 8.4 in the smallest call.  A block joined by the CTA that comes last instead of by a second
//     kernel: 197 us, and 8 x 1 token over ~750 positions 17.3 us for 15.0.
//   1 token over 4098 positions                 15 us, 8 of them before the first
//     product and in the join
#include <cmath>
#include <limits>
#include <type_traits>

#include <cuda.h>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 384;
// registers per thread: the launch gives every thread 168; the warpgroup of
// warps 8-11 gives up most of its own and the softmax warpgroups share them
// (256 * 208 + 128 * 88 = 384 * 168)
constexpr int kSoftmaxRegs = 208;
constexpr int kIssueRegs = 88;
constexpr int kCtas = 152;              // at most: the workspace does not depend on the device
constexpr int kHalfRows = 128;
constexpr int kBlockRows = 2 * kHalfRows;
constexpr int kTile = 128;              // cache positions per tile
constexpr int kColBytes = 128;          // one swizzle span: 64 elements
constexpr int kHalfTileBytes = kTile * kColBytes;    // 128 rows of 64 elements
constexpr int kRingBytes = 10 * kHalfTileBytes;      // 160 KiB of K / V stages
constexpr float kRescale = 8.f;         // growth of the maximum (in log2) that moves m
constexpr uint32_t kTmemCols = 512;     // S0 | S1 | O0 | O1
constexpr uint32_t kProducers = 2;      // warps 8 and 11, which take the loads in turn
constexpr long long kDrainLimit = 1ll << 31;
constexpr long long kProbeCycles = 1ll << 20;

struct AttendParams {
  const void* q;
  void* out;
  float* lse;
  long long q_ts, q_hs, o_ts, o_hs;
  int Hq, Hkv, G, D, T, B, N, MW;
  FastDiv by_group, by_page;
  const int32_t* lengths;
  const int32_t* starts;
  const uint32_t* mask;
  float c;                    // |scale| log2 e
  uint32_t negate;            // the products of Q and K change their sign: the scale is negative
  bool wide_out;              // 32-byte stores
  const int32_t* table;
  long long table_stride;
  long long cap;              // positions a sequence's pages can hold
  int page, pages, box;       // positions per page, pages, positions per TMA box
  int k_slot[3], v_slot[3];   // which of (head, row, page) is coordinate 1, 2, 3
  const void* v;              // the values again, for what a product cannot take (see take_out)
  long long v_ps, v_rs, v_hs;
  uint32_t* err;
  struct Joint* joints;       // [kCtas]
  float4* parts;              // [kCtas][2] slots: [cols / 4][slot_rows] float4, then [slot_rows] (m, l)
  int slot_rows;
  long long wait_limit;
};

// A block of rows whose tiles ended in a later CTA than they began in.
struct Joint {
  int parts;                  // CTAs that share it, this one the first; 0 = none
  int rows, row0;             // rows of the block, its first row within (sequence, head)
  int head, token0;           // key head, the sequence's first token
  int pad[3];
};

// A CTA's slot 1 takes the block that begins in it and goes on in the next one,
// slot 0 a block that began before it.
template <int COLS>
__device__ __forceinline__ float4* part_slot(const AttendParams& P, int cta, int slot) {
  return P.parts + (long long)(2 * cta + slot) * ((COLS / 4) * P.slot_rows + (P.slot_rows + 1) / 2);
}

// ----------------------------------------------------------------- PTX glue
__device__ __forceinline__ void tma_box(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      :: "r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               :: "r"(smem_u32(bar)) : "memory");
}
// One thread of the warp issues; the warp runs converged so that descriptors
// and addresses stay in uniform registers.
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
               :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
               :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float* x) {
  uint32_t* r = reinterpret_cast<uint32_t*>(x);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes in
// groups of 8 (1024 bytes apart: the stride offset); `lead` is the distance
// between blocks of 64 columns where the 64-element span runs along the
// operand's outer dimension (V), and unused where it runs along K (Q, K).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 32 bytes (32-byte aligned) in one store.
__device__ __forceinline__ void stg_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 16 bytes from memory (or zeros) to shared memory, without a register.
__device__ __forceinline__ void cp_async16_or_zero(void* dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               :: "r"(smem_u32(dst)), "l"(src), "r"(copy ? 16u : 0u) : "memory");
}

// The log-sum-exp of a row with maximum m (of c S) and sum l: -inf where it sees nothing, NaN stays NaN.
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// Operand type in the instruction descriptor.
template <typename T> constexpr uint32_t kTypeCode = 0;
template <> constexpr uint32_t kTypeCode<__nv_bfloat16> = 1;

// TMEM loads fill registers asynchronously: after this wait the N values of x
// are there, and the compiler may not have used them before.
template <int N>
__device__ __forceinline__ void loaded(float* x) {
  tc_wait_ld();
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+f"(x[k]));
}

// ----------------------------------------------------------------- the work
// One sequence's chunk.
struct Chunk {
  int start, n, len, lead, S, rows, blocks;       // rows = n * G < 2^31
};
__device__ __forceinline__ Chunk load_chunk(const AttendParams& P, int b) {
  Chunk c;
  const int s0 = P.starts[b], s1 = min(P.starts[b + 1], P.T);
  c.start = s0;
  c.n = s0 >= 0 && s1 > s0 ? s1 - s0 : 0;
  c.len = int(min((long long)max(P.lengths[b], 0), P.cap));
  c.S = int(min((long long)c.len + c.n, P.cap));
  c.lead = max(c.n - P.N, 0);
  c.rows = c.n * P.G;
  c.blocks = int((unsigned(c.rows) + kBlockRows - 1) / kBlockRows);
  return c;
}
// Positions that some row of block `blk` sees end here.
__device__ __forceinline__ int block_end(const AttendParams& P, const Chunk& c, int blk) {
  const int r1 = c.rows - blk * kBlockRows < kBlockRows ? c.rows : (blk + 1) * kBlockRows;
  const int last = P.by_group.div(r1 - 1);
  return last >= c.lead ? c.S : min(c.len + last + 1, c.S);
}
__device__ __forceinline__ int block_tiles(const AttendParams& P, const Chunk& c, int blk) {
  return max(1, (block_end(P, c, blk) + kTile - 1) / kTile);
}
// Tiles of all blocks of one head.
__device__ __forceinline__ long long head_tiles(const AttendParams& P, const Chunk& c) {
  if (c.blocks == 0) return 0;
  long long t = 0;
  // blocks of nodes and the last one see everything; causal ones less
  for (int k = 0; k < c.blocks; ++k) {
    const int n = block_tiles(P, c, k);
    if (P.by_group.div(k * kBlockRows) >= c.lead) return t + (long long)n * (c.blocks - k);
    t += n;
  }
  return t;
}

// A CTA's walk over its span of the tile list, a block's part at a time.
struct Walk {
  int left;                   // tiles of the span from this part on
  int b, h, blk;              // the block
  Chunk c;
  int tiles, end, rows;       // of the block: its tiles, where the last one ends, its rows
  int t0, t1;                 // the part: tiles t0 .. t1 in the order in which they are taken

  // Every other block takes its tiles from the last to the first: the ones that the
  // block before it, over the same cache, has just read are still in L2 (2 x 2048
  // tokens over 32768 positions 1363 -> 1337 us, 64 trees of 79 rows 187 -> 185.5).
  __device__ __forceinline__ int tile(int t) const { return blk & 1 ? tiles - 1 - t : t; }
  __device__ __forceinline__ void open(const AttendParams& P, int from) {
    tiles = block_tiles(P, c, blk);
    end = block_end(P, c, blk);
    rows = min(kBlockRows, c.rows - blk * kBlockRows);
    t0 = from;
    t1 = min(tiles, from + left);
  }
  __device__ __forceinline__ bool next(const AttendParams& P) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++blk >= c.blocks) {
      blk = 0;
      if (++h >= P.Hkv) {
        h = 0;
        do {
          if (++b >= P.B) return false;
          c = load_chunk(P, b);
        } while (c.blocks == 0);
      }
    }
    open(P, 0);
    return true;
  }
};

// What the CTA's span is, and where it begins.
struct Span {
  long long total, u0, u1, base;   // base: the first tile of sequence b
  int b, ctas;
};

struct Shared {
  uint64_t kv_full[10], kv_empty[10];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drain[2];
  Span span;
  long long scan[kThreads / 32];
  uint32_t tmem;
  int dead;                        // a wait ran out: everyone leaves
  int odd;                         // a row whose block's rows see different positions is not finite
};

// Bounded wait of a whole warp; false (for all lanes) once any wait of the CTA ran
// out.  A probe may suspend the thread for some microseconds, so a limit below
// that (a test of this path) is kept by probes that do not.
__device__ __forceinline__ bool wait_lane(uint64_t* bar, uint32_t parity, Shared* sh, long long limit) {
  if (mbar_test_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!(limit < kProbeCycles ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
    if (*reinterpret_cast<volatile int*>(&sh->dead)) return false;
    if (clock64() - t0 > limit) {
      *reinterpret_cast<volatile int*>(&sh->dead) = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Shared* sh, long long limit) {
  return __all_sync(kFull, wait_lane(bar, parity, sh, limit));
}

// x * c / n for c <= n <= kCtas.
__device__ __forceinline__ long long share(long long x, int c, int n) {
  if (x < (1ll << 24)) return (unsigned(x) * unsigned(c)) / unsigned(n);
  return x * c / n;
}

// All threads: the tile count of all sequences, this CTA's span and the
// sequence it begins in.  Sequences are taken kThreads at a time; when they fit
// in one such group its scan is kept, else a second pass looks for the span.
__device__ void find_span(const AttendParams& P, Shared* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  const bool one_group = P.B <= kThreads;
  long long before = 0, cost = 0, incl = 0;
  bool bad = false;
  auto scan = [&](int b) {           // cost of sequence b, the inclusive sum in incl, the group's total added to before
    cost = 0;
    if (b < P.B) {
      const Chunk c = load_chunk(P, b);
      cost = head_tiles(P, c) * P.Hkv;
      bad |= P.lengths[b] < 0 || (c.n > 0 && (long long)P.lengths[b] + c.n > P.cap);
    }
    incl = cost;
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) sh->scan[warp] = incl;
    __syncthreads();
    long long lower = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long x = sh->scan[w];
      if (w < warp) lower += x;
      before += x;
    }
    incl += lower;
  };
  auto locate = [&](int b, long long u0) {
    if (cost > 0 && u0 >= incl - cost && u0 < incl) {
      sh->span.b = b;
      sh->span.base = incl - cost;
    }
  };
  for (int b0 = 0; b0 < P.B; b0 += kThreads) scan(b0 + tid);
  const long long total = before;
  const int ctas = int(min((long long)gridDim.x, total)), c = blockIdx.x;
  const long long u0 = c < ctas ? share(total, c, ctas) : total;
  const long long u1 = c < ctas ? share(total, c + 1, ctas) : total;
  if (tid == 0) {
    sh->span.total = total;
    sh->span.ctas = ctas;
    sh->span.u0 = u0;
    sh->span.u1 = u1;
  }
  if (one_group) {
    locate(tid, u0);
  } else {
    before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      scan(b0 + tid);
      locate(b0 + tid, u0);
    }
  }
  if (bad && blockIdx.x == 0) set_dev_error(P.err, DART_DEVERR_CACHE);
}

__device__ __forceinline__ bool begin_walk(const AttendParams& P, const Shared* sh, Walk& w) {
  w.left = int(sh->span.u1 - sh->span.u0);
  if (w.left <= 0) return false;
  w.b = sh->span.b;
  w.c = load_chunk(P, w.b);
  const long long per_head = head_tiles(P, w.c);
  long long off = sh->span.u0 - sh->span.base;
  if (off < (1ll << 31) && per_head < (1ll << 31)) w.h = int(unsigned(off) / unsigned(per_head));
  else w.h = int(off / per_head);
  off -= w.h * per_head;
  w.blk = 0;
  for (;;) {
    const int n = block_tiles(P, w.c, w.blk);
    if (n > off || w.blk + 1 >= w.c.blocks) break;
    off -= n;
    ++w.blk;
  }
  w.open(P, int(off));
  return true;
}

// Loads of a part of n tiles enter the ring as K0, then K(j+1) and V(j) in turn.
__device__ __forceinline__ int k_load(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_load(int j, int n) { return j < n - 1 ? 2 * j + 2 : 2 * n - 1; }

// A row's P is 0 where it does not see, but 0 * NaN is NaN in the product: where a
// block's rows see different positions, an infinity or NaN in V reaches rows that
// it must not reach.  A row finds that in its sums at the block's end; the CTA then
// goes over its span once more, carefully: what is not finite is taken out of those
// tiles before the product and given back to the rows that see it.  (Looking at the
// tiles themselves, every time, cost a tenth: the products need the shared memory.)
// take_out: the threads of a half go over the tile's `valid` rows; both halves write
// the same.
template <typename T> constexpr uint32_t kExpBits = 0x7F807F80u;
template <> constexpr uint32_t kExpBits<__half> = 0x7C007C00u;
template <typename T, int DH>
__device__ __forceinline__ void take_out(unsigned char* v, int valid) {
  constexpr uint32_t e = kExpBits<T>, one = e & (0u - e) & 0xFFFFu;
  unsigned char* mine = v + (threadIdx.x & 127) * 16;           // eight threads a row
  const int r0 = (threadIdx.x & 127) >> 3;
#pragma unroll 1
  for (int i = 0; i < 8 * DH; ++i)
    if (16 * (i & 7) + r0 < valid) {
      uint32_t* x = reinterpret_cast<uint32_t*>(mine + i * 2048);
      for (int k = 0; k < 4; ++k) {
        // the top bit of each element whose exponent is all ones
        const uint32_t odd = ((x[k] & e) + (one | one << 16)) & 0x80008000u;
        if (odd) x[k] &= ~((odd >> 15) * 0xFFFFu);
      }
    }
  fence_async();
}
// Between the passes: true if there is a second one.  Once per thread of the CTA.
__device__ __forceinline__ bool go_over_again(const Shared* sh) {
  asm volatile("bar.sync 1, %0;" :: "n"(kThreads) : "memory");
  return __all_sync(kFull, *reinterpret_cast<const volatile int*>(&sh->odd) != 0 &&
                               *reinterpret_cast<const volatile int*>(&sh->dead) == 0);
}

template <typename T, int DH>       // DH: blocks of 64 columns per head
__global__ void __launch_bounds__(kThreads, 1)
attend_kernel(const AttendParams P, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  constexpr int kStageBytes = DH * kHalfTileBytes;
  constexpr int kStages = kRingBytes / kStageBytes;
  constexpr int kCols = 64 * DH;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* sq = smem;                               // 2 halves of Q
  unsigned char* ring = smem + 2 * kStageBytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + kRingBytes);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh->kv_full[i], 1);
      mbar_init(&sh->kv_empty[i], 2);        // one from either half
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->q_full[t], 4);
      mbar_init(&sh->s_full[t], 1);
      mbar_init(&sh->p_full[t], 4);
      mbar_init(&sh->o_full[t], 1);
    }
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    fence_mbar_init();
    sh->dead = 0;
    sh->odd = 0;
    P.joints[blockIdx.x].parts = 0;        // this thread names the CTA's joint later, if there is one
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  __syncthreads();
  find_span(P, sh);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = sh->tmem;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssueRegs));
    if (warp == 8 || warp == 11) {
      // ------------------------------------------------------------ producers
      const uint32_t pid = warp == 8 ? 0u : 1u;
      uint32_t idx = 0, turn = 0;            // loads so far, and whose turn the next one is
      bool ok = true;
      auto span_of = [&]() {
        Walk w;
        bool more = begin_walk(P, sh, w);
        while (more && ok) {
          const int n = w.t1 - w.t0;
          const int32_t* table = P.table + (long long)w.b * P.table_stride;
          for (int i = 0; i < 2 * n && ok; ++i, ++idx) {
            if (turn != pid) {
              turn = turn + 1 < kProducers ? turn + 1 : 0;
              continue;
            }
            turn = turn + 1 < kProducers ? turn + 1 : 0;
            const bool is_k = i == 0 || (i < 2 * n - 1 && (i & 1));
            const int j = is_k ? (i + 1) / 2 : (i == 2 * n - 1 ? n - 1 : (i - 2) / 2);
            const int p0 = w.tile(w.t0 + j) * kTile;
            const int boxes = (min(w.end - p0, kTile) + P.box - 1) / P.box;      // 0 for a block that sees nothing
            const int at = p0 + (lane / DH) * P.box;
            const bool mine = lane / DH < boxes;
            int page = 0;
            if (mine) {
              page = table[P.by_page.div(at)];
              if (page < 0 || page >= P.pages) {
                set_dev_error(P.err, DART_DEVERR_CACHE);
                page = P.pages;               // out of the map's range: the box arrives as zeros
              }
            }
            const uint32_t stage = idx % kStages;
            ok = wait_warp(&sh->kv_empty[stage], ((idx / kStages) & 1u) ^ 1u, sh, P.wait_limit);
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(&sh->kv_full[stage], uint32_t(boxes * DH * P.box * kColBytes));
            __syncwarp();
            if (mine) {
              const int half = lane % DH, row = at - P.by_page.div(at) * P.page;
              const int* slot = is_k ? P.k_slot : P.v_slot;
              auto pick = [&](int i) { return slot[i] == 0 ? w.h : slot[i] == 1 ? row : page; };
              tma_box(ring + stage * kStageBytes + half * kHalfTileBytes + (lane / DH) * P.box * kColBytes,
                      is_k ? &kmap : &vmap, 64 * half, pick(0), pick(1), pick(2),
                      &sh->kv_full[stage]);
            }
          }
          if (ok) more = w.next(P);
        }
      };
      span_of();
      if (go_over_again(sh)) span_of();
      // no copy may land after the CTA has left: the last load of each stage is waited for
      for (uint32_t i = idx > uint32_t(kStages) ? idx - kStages : 0; i < idx; ++i)
        if (i % kProducers == pid) mbar_wait_bounded(&sh->kv_full[i % kStages], (i / kStages) & 1u, kDrainLimit);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- tensor unit
      constexpr uint32_t type = kTypeCode<T>;
      constexpr uint32_t id_s = (1u << 4) | (type << 7) | (type << 10) | (uint32_t(kTile >> 3) << 17) |
                                (uint32_t(kHalfRows >> 4) << 24);
      constexpr uint32_t id_o = (1u << 4) | (type << 7) | (type << 10) | (1u << 16) | (uint32_t(kCols >> 3) << 17) |
                                (uint32_t(kHalfRows >> 4) << 24);
      const uint64_t q_desc = smem_desc(smem_u32(sq), 16), k_desc = smem_desc(smem_u32(ring), 16),
                     v_desc = smem_desc(smem_u32(ring), kHalfTileBytes);
      const int k_steps = (P.D + 15) / 16;
      const int t = warp - 9;                 // the half whose products this warp issues
      const uint32_t s_at = tmem + t * kTile, o_at = tmem + 2 * kTile + t * kCols;
      const uint64_t qd = q_desc + t * (kStageBytes >> 4);
      uint32_t idx = 0, q_seen = 0, p_seen = 0;
      bool ok = true;
      auto span_of = [&]() {
        Walk w;
        bool more = begin_walk(P, sh, w);
        while (more && ok) {
          const int n = w.t1 - w.t0;
          if (w.rows <= t * kHalfRows) {
            // The block has no second half.  This warp still sees every load arrive
            // and gives its stage up: a stage's phases are told apart by their
            // parity alone, so nobody may fall two of them behind or run ahead.
            for (int i = 0; i < 2 * n && ok; ++i, ++idx) {
              ok = wait_warp(&sh->kv_full[idx % kStages], (idx / kStages) & 1u, sh, P.wait_limit);
              if (ok && lane == 0) mbar_arrive(&sh->kv_empty[idx % kStages]);
            }
            if (ok) more = w.next(P);
            continue;
          }
          for (int j = -1; j < n; ++j) {
            uint32_t ks = 0, vs = 0;
            if (j + 1 < n) {
              const uint32_t i = idx + k_load(j + 1);
              ks = i % kStages;
              if (!(ok = wait_warp(&sh->kv_full[ks], (i / kStages) & 1u, sh, P.wait_limit))) break;
            }
            if (j >= 0) {
              const uint32_t i = idx + v_load(j, n);
              vs = i % kStages;
              if (!(ok = wait_warp(&sh->kv_full[vs], (i / kStages) & 1u, sh, P.wait_limit))) break;
            }
            // steps of 16 positions; those wholly behind the block's end are left out
            const int steps = max(1, (min(w.end - w.tile(w.t0 + j) * kTile, kTile) + 15) / 16);
            ok = j < 0 ? wait_warp(&sh->q_full[t], q_seen++ & 1u, sh, P.wait_limit)
                       : wait_warp(&sh->p_full[t], p_seen++ & 1u, sh, P.wait_limit);
            if (!ok) break;
            tc_after();
            if (elect()) {
              if (j >= 0) {
                const uint64_t vd = v_desc + uint64_t(vs * (kStageBytes >> 4));
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                  if (k < steps) mma_ts(o_at, s_at + k * 8, vd + k * (16 * kColBytes >> 4), id_o, j > 0 || k > 0);
              }
              if (j + 1 < n) {
                const uint64_t kd = k_desc + uint64_t(ks * (kStageBytes >> 4));
#pragma unroll
                for (int k = 0; k < 4 * DH; ++k) {
                  const int off = ((k >> 2) * kHalfTileBytes + (k & 3) * 32) >> 4;
                  if (k < k_steps) mma_ss(s_at, qd + off, kd + off, id_s | P.negate, k > 0);
                }
              }
              tc_commit(j + 1 < n ? &sh->s_full[t] : &sh->o_full[t]);
              if (j >= 0) tc_commit(&sh->kv_empty[vs]);
              if (j + 1 < n) tc_commit(&sh->kv_empty[ks]);
            }
            __syncwarp();
          }
          idx += 2 * n;
          if (ok) more = w.next(P);
        }
      };
      span_of();
      if (go_over_again(sh)) span_of();
      // every product has ended before the tensor memory is given back
      if (elect()) tc_commit(&sh->drain[t]);
      mbar_wait_bounded(&sh->drain[t], 0, kDrainLimit);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;                       // within the half
    const uint32_t lane_base = uint32_t(warp & 3) << 21;          // TMEM lanes 32 (warp & 3) ..
    const uint32_t ts = tmem + lane_base + uint32_t(t) * kTile;
    const uint32_t to = tmem + lane_base + 2 * kTile + uint32_t(t) * kCols;
    unsigned char* q_half = sq + t * kStageBytes;
    uint32_t idx = 0, s_seen = 0, o_seen = 0;
    bool ok = true;

    auto span_of = [&](auto careful) {
      constexpr bool kCareful = decltype(careful)::value;
      Walk w;
      bool more = begin_walk(P, sh, w);
      auto active = [&]() { return w.rows > t * kHalfRows; };
      auto skip_inactive = [&]() {
        while (more && !active()) {
          idx += 2 * (w.t1 - w.t0);
          more = w.next(P);
        }
      };
      // This warp's 32 rows of the block's queries, swizzled, copied without registers
      // as soon as the buffer is free; give_q hands them to the products.  Lane r finds
      // where row r lies (when each lane found its vector's row, step by step, a block
      // took 2600 cycles to ask).
      constexpr int kChunks = 8 * DH, kPer = 32 / kChunks;        // 16-byte chunks a row, rows a step
      auto ask_q = [&]() {
        const int chunk = lane % kChunks, sub = lane / kChunks, first = (warp & 3) * 32;
        const int rows = w.rows - t * kHalfRows - first;
        const int g = w.blk * kBlockRows + t * kHalfRows + first + max(0, min(lane, rows - 1));
        const int token = P.by_group.div(g);
        const long long at = (long long)(w.c.start + token) * P.q_ts + (long long)(w.h * P.G + g - token * P.G) * P.q_hs;
        const bool inside = 8 * chunk < P.D;
        const T* src = static_cast<const T*>(P.q) + (inside ? 8 * chunk : 0);
        unsigned char* dst = q_half + (chunk >> 3) * kHalfTileBytes + first * kColBytes;
#pragma unroll 4
        for (int u = 0; u < 32 / kPer; ++u) {
          const int r = u * kPer + sub;
          const long long from = __shfl_sync(kFull, at, r);
          if (r < rows) cp_async16_or_zero(dst + r * kColBytes + (((chunk & 7) ^ (r & 7)) << 4), src + from, inside);
        }
        cp_async_commit();
      };
      auto give_q = [&]() {
        cp_async_wait<0>();
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_full[t]);
      };

      skip_inactive();
      if (more) {
        ask_q();
        give_q();
      }
      while (more && ok) {
        const int n = w.t1 - w.t0;
        const int my_row = t * kHalfRows + row;
        const bool warp_on = t * kHalfRows + (warp & 3) * 32 < w.rows;
        const bool row_on = my_row < w.rows;
        const int g = w.blk * kBlockRows + min(my_row, w.rows - 1);
        const int token = P.by_group.div(g);
        // the row sees positions below `plain` and the set bits from `tree` on
        const int plain = min(w.c.len + min(token + 1, w.c.lead), w.c.S);
        const int tree = w.c.len + w.c.lead;
        const int nodes = token >= w.c.lead ? min(min(P.N, w.c.n - w.c.lead), w.c.S - tree) : 0;   // may be < 0
        const uint32_t* bits = P.mask + ((long long)w.b * P.N + (token - w.c.lead)) * P.MW;    // read if nodes > 0
        // tiles below the block's least `plain` need no mask
        const int first_token = P.by_group.div(w.blk * kBlockRows);
        const int open_end = min(w.c.len + min(first_token + 1, w.c.lead), w.c.S);

        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < n && ok; ++j) {
          const int tile = w.tile(w.t0 + j), p0 = tile * kTile;
          // what this row sees of the tile, looked up while the product is under way
          const bool masked = p0 + kTile > open_end;
          uint32_t see[4] = {kFull, kFull, kFull, kFull};
          if (masked) {
            uint32_t word[5];
            const int at0 = p0 - tree, wd0 = at0 >> 5;           // floor: the word that holds bit at0
#pragma unroll
            for (int i = 0; i < 5; ++i)
              word[i] = wd0 + i >= 0 && 32 * (wd0 + i) < nodes ? bits[wd0 + i] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int below = max(0, min(plain - p0 - 32 * i, 32)), left = max(0, min(nodes - at0 - 32 * i, 32));
              const uint32_t x = __funnelshift_r(word[i], word[i + 1], at0 & 31);
              see[i] = (below >= 32 ? kFull : (1u << below) - 1u) | (x & (left >= 32 ? kFull : (1u << left) - 1u));
            }
          }
          ok = wait_warp(&sh->s_full[t], s_seen++ & 1u, sh, P.wait_limit);
          if (!ok) break;
          if (kCareful && masked && open_end < w.end) {
            const uint32_t i = idx + v_load(j, n);
            ok = wait_warp(&sh->kv_full[i % kStages], (i / kStages) & 1u, sh, P.wait_limit);
            if (!ok) break;
            take_out<T, DH>(ring + (i % kStages) * kStageBytes, min(w.end - p0, kTile));
          }
          tc_after();
          if (warp_on) {
            float s[kTile];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s + 32 * i);
            loaded<kTile>(s);
            if (masked) {
#pragma unroll
              for (int k = 0; k < kTile; ++k)
                if (!((see[k >> 5] >> (k & 31)) & 1u)) s[k] = -INFINITY;
            }
            float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k < kTile; k += 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                top[i] = k + 4 + i < kTile ? max3(top[i], s[k + i], s[k + 4 + i]) : fmaxf(top[i], s[k + i]);
            }
            float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            mx *= P.c;
            if (j == 0) {
              m = mx;
            } else {
              const bool grow = mx > m + kRescale;
              if (__any_sync(kFull, grow)) {
                const float keep = grow ? ex2_approx(m - mx) : 1.f;
                if (grow) {
                  m = mx;
                  l *= keep;
                }
#pragma unroll
                for (int i = 0; i < kCols / 16; ++i) {
                  float o[16];
                  tmem_ld16(to + 16 * i, o);
                  loaded<16>(o);
#pragma unroll
                  for (int k = 0; k < 16; ++k) o[k] *= keep;
                  tmem_st16(to + 16 * i, reinterpret_cast<const uint32_t*>(o));
                }
              }
            }
            const float off = m == -INFINITY ? 0.f : m;
            const uint64_t c2 = pair(P.c, P.c), off2 = pair(-off, -off);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t pk[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const uint64_t x = fma2(pair(s[32 * i + 2 * k], s[32 * i + 2 * k + 1]), c2, off2);
                const float a = ex2_approx(low(x)), b = ex2_approx(high(x));
                sum[k & 1] = add2(sum[k & 1], pair(a, b));
                pk[k] = pack2<T>(a, b);
              }
              tmem_st16(ts + 16 * i, pk);
            }
            sum[0] = add2(sum[0], sum[1]);
            l += low(sum[0]) + high(sum[0]);
            tc_wait_st();
          }
          // V rows behind the end may hold anything, and 0 * NaN is NaN: those that
          // share a step of 16 with valid rows are cleared (by either half, which write the same)
          if (tile == w.tiles - 1) {
            const int valid = max(0, min(w.end - p0, kTile));
            const int upto = max(16, (valid + 15) / 16 * 16);
            if (valid < upto) {
              const uint32_t i = idx + v_load(j, n);
              ok = wait_warp(&sh->kv_full[i % kStages], (i / kStages) & 1u, sh, P.wait_limit);
              if (!ok) break;
              const int r = valid + ((tid & 127) >> 3);
              if (r < upto)
#pragma unroll
                for (int hf = 0; hf < DH; ++hf)
                  *reinterpret_cast<uint4*>(ring + (i % kStages) * kStageBytes + hf * kHalfTileBytes + r * kColBytes +
                                            (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_async();
            }
          }
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->p_full[t]);
        }
        if (!ok) break;
        idx += 2 * n;

        // the finished part, while the next one's queries are already on their way
        const int d_start = w.c.start, d_h = w.h, d_row0 = w.blk * kBlockRows, d_rows = w.rows, d_t0 = w.t0;
        const int d_after = w.tiles - w.t1;                // the block's tiles in later CTAs
        const int tile0 = min(w.tile(w.t0), w.tile(w.t1 - 1)), d_b = w.b;
        const int d_odd0 = open_end < w.end ? max(open_end / kTile, tile0) * kTile : w.end;
        const int d_odd1 = min((tile0 + n) * kTile, w.end);      // rows differ in what they see of d_odd0 .. d_odd1
        more = w.next(P);
        skip_inactive();
        if (more) ask_q();
        ok = wait_warp(&sh->o_full[t], o_seen++ & 1u, sh, P.wait_limit);
        if (!ok) break;
        tc_after();
        const bool differ = d_odd0 < d_odd1;
        uint64_t odd = 0ull;                               // 0 while all is finite, else NaN
        auto look = [&](const float* o) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) odd = fma2(pair(o[k], o[k + 1]), 0ull, odd);
        };
        if (kCareful && differ && warp_on) {         // what take_out took is given to the rows that see it
          const int32_t* table = P.table + (long long)d_b * P.table_stride;
#pragma unroll 1
          for (int col = 0; col < P.D; col += 8) {
            float o[8];
            tmem_ld8(to + col, o);
            loaded<8>(o);
#pragma unroll 1
            for (int p = d_odd0; p < d_odd1; ++p) {
              const int x = p - tree, pg = P.by_page.div(p), page = table[pg];
              const bool sees = p < plain || (x >= 0 && x < nodes && (bits[x >> 5] >> (x & 31) & 1u));
              if (!sees || page < 0 || page >= P.pages) continue;
              const T* src = static_cast<const T*>(P.v) + page * P.v_ps + (p - pg * P.page) * P.v_rs + d_h * P.v_hs;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float y = float(src[col + k]);
                if (!(fabsf(y) < INFINITY)) o[k] += y;
              }
            }
            __syncwarp();
            tmem_st8(to + col, reinterpret_cast<const uint32_t*>(o));
          }
          tc_wait_st();
        }
        if (d_t0 == 0 && d_after == 0) {
          // A thread's row leaves 32 (or 16) bytes at a time: whole sectors, and
          // nothing to wait for.  (Through shared memory the rows would leave in
          // whole lines, but the next queries would have to wait for the buffer.)
          const float inv = l > 0.f ? 1.f / l : 0.f;
          if (warp_on) {
            const long long tok = d_start + token;
            const int head = d_h * P.G + g - token * P.G;
            T* dst = static_cast<T*>(P.out) + tok * P.o_ts + (long long)head * P.o_hs;
#pragma unroll
            for (int i = 0; i < kCols / 32; ++i) {
              float o[32];
              tmem_ld32(to + 32 * i, o);
              loaded<32>(o);
              if (!kCareful) look(o);
              uint32_t y[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = pack2<T>(o[2 * k] * inv, o[2 * k + 1] * inv);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                T* to_row = dst + 32 * i + 16 * k;
                // (305 us for 314 with 16 bytes, 2 x 1024 tokens over 16384 positions)
                if (P.wide_out) {
                  if (row_on && 32 * i + 16 * k < P.D) stg_v8(to_row, y + 8 * k);
                } else {
                  if (row_on && 32 * i + 16 * k < P.D)
                    *reinterpret_cast<uint4*>(to_row) = make_uint4(y[8 * k], y[8 * k + 1], y[8 * k + 2], y[8 * k + 3]);
                  if (row_on && 32 * i + 16 * k + 8 < P.D)
                    *reinterpret_cast<uint4*>(to_row + 8) =
                        make_uint4(y[8 * k + 4], y[8 * k + 5], y[8 * k + 6], y[8 * k + 7]);
                }
              }
              if (i == 0 && more) give_q();
            }
            if (row_on && P.lse) P.lse[tok * P.Hq + head] = log_sum(m, l);
          }
        } else if (warp_on) {
          // [4 columns][row] so that a warp writes whole lines, then (m, l) of each row
          float4* dst = part_slot<kCols>(P, blockIdx.x, d_t0 > 0 ? 0 : 1);
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i) {
            float o[32];
            tmem_ld32(to + 32 * i, o);
            loaded<32>(o);
            if (!kCareful) look(o);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (row_on)
                dst[(8 * i + k) * P.slot_rows + my_row] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            if (i == 0 && more) give_q();
          }
          if (row_on) reinterpret_cast<float2*>(dst + kCols / 4 * P.slot_rows)[my_row] = make_float2(m, l);
        }
        if (!kCareful && odd != 0ull && differ && row_on) *reinterpret_cast<volatile int*>(&sh->odd) = 1;
        if (!warp_on && more) give_q();
        if (t == 0 && warp == 0 && lane == 0 && d_t0 == 0 && d_after > 0) {
          // the span ends within the block: the joint names it and the CTAs that share it
          const Span& sp = sh->span;
          Joint jt;
          jt.parts = int(((sp.u1 + d_after) * sp.ctas - 1) / sp.total) - int(blockIdx.x) + 1;
          jt.rows = d_rows;
          jt.row0 = d_row0;
          jt.head = d_h;
          jt.token0 = d_start;
          P.joints[blockIdx.x] = jt;
        }
      }
    };
    span_of(std::false_type{});
    if (go_over_again(sh)) span_of(std::true_type{});
  }

  tc_before();
  __syncthreads();
  tc_after();
  if (warp == 9) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols));
    if (lane == 0 && sh->dead) set_dev_error(P.err, DART_DEVERR_WAIT_TIMEOUT);
  }
}

// Rows of a block whose tiles several CTAs shared, in one pass over the parts:
//   m = max m_i,  l = sum l_i 2^(m_i - m),  out = (sum O_i 2^(m_i - m)) / l
// Latency bounds it, so nothing waits for another thread: a thread takes four
// columns of two rows and four parts at a time, and finds its rows' weights
// itself.  A warp covers 8 rows by 4 column groups, so that the parts (16 bytes
// of 8 rows) and the output (8 bytes of 4 groups) move in whole sectors.
constexpr int kJoinRows = 16, kJoinBatch = 4;
template <typename T, int DH>
__global__ void __launch_bounds__(128 * DH)
join_kernel(const AttendParams P) {
  constexpr int kCols = 64 * DH, kC4 = kCols / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Joint jt = P.joints[blockIdx.x];
  const int r0 = blockIdx.y * kJoinRows + (threadIdx.x & 7), c4 = threadIdx.x >> 3;
  if (jt.parts <= 0 || r0 >= jt.rows) return;
  const bool two = r0 + 8 < jt.rows;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = 0; i0 < jt.parts; i0 += kJoinBatch) {
    float4 x[kJoinBatch][2];
    float2 ml[kJoinBatch][2];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ml[i][e] = make_float2(-INFINITY, 0.f);
        x[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i0 + i < jt.parts && (e == 0 || two)) {
          const float4* slot = part_slot<kCols>(P, blockIdx.x + i0 + i, i0 + i == 0 ? 1 : 0);
          ml[i][e] = reinterpret_cast<const float2*>(slot + kC4 * P.slot_rows)[r0 + 8 * e];
          x[i][e] = slot[c4 * P.slot_rows + r0 + 8 * e];
        }
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = m[e];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) top = fmaxf(top, ml[i][e].x);
      const float off = top == -INFINITY ? 0.f : top;
      const float keep = ex2_approx(m[e] - off);
      m[e] = top;
      l[e] *= keep;
      acc[e].x *= keep;
      acc[e].y *= keep;
      acc[e].z *= keep;
      acc[e].w *= keep;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        const float f = ex2_approx(ml[i][e].x - off);
        l[e] = fmaf(ml[i][e].y, f, l[e]);
        acc[e].x = fmaf(x[i][e].x, f, acc[e].x);
        acc[e].y = fmaf(x[i][e].y, f, acc[e].y);
        acc[e].z = fmaf(x[i][e].z, f, acc[e].z);
        acc[e].w = fmaf(x[i][e].w, f, acc[e].w);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (e == 1 && !two) break;
    const float inv = l[e] > 0.f ? 1.f / l[e] : 0.f;
    const int g = jt.row0 + r0 + 8 * e, token = P.by_group.div(g);
    const long long tok = jt.token0 + token;
    const int head = jt.head * P.G + g - token * P.G;
    if (4 * c4 < P.D)
      *reinterpret_cast<uint2*>(static_cast<T*>(P.out) + tok * P.o_ts + (long long)head * P.o_hs + 4 * c4) =
          make_uint2(pack2<T>(acc[e].x * inv, acc[e].y * inv), pack2<T>(acc[e].z * inv, acc[e].w * inv));
    if (P.lse && c4 == 0) P.lse[tok * P.Hq + head] = log_sum(m[e], l[e]);
  }
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }
bool mult8(long long a, long long b) { return ((a | b) & 7) == 0; }
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn tensor_map_encoder() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (settled(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q)) !=
            cudaSuccess || q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// The cache as a 4-dimensional map (columns, then head, row and page in the
// order of their strides) with a box of `box` rows by 64 columns; slot[i]
// names what coordinate i + 1 is: 0 head, 1 row, 2 page.
bool cache_map(const dart_cache_t& c, const void* base, long long page_stride, long long row_stride,
               long long head_stride, int box, CUtensorMap* map, int* slot) {
  const EncodeFn encode = tensor_map_encoder();
  if (!encode) return false;
  const long long size[3] = {c.heads, c.page, c.pages};
  const long long stride[3] = {head_stride, row_stride, page_stride};
  for (int i = 0; i < 3; ++i) slot[i] = i;
  auto key = [&](int i) { return size[i] > 1 ? stride[i] : -1ll; };     // dimensions of one come first
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (key(slot[j]) > key(slot[j + 1])) {
        const int x = slot[j];
        slot[j] = slot[j + 1];
        slot[j + 1] = x;
      }
  cuuint64_t dims[4] = {cuuint64_t(c.dim), 0, 0, 0}, strides[3];
  cuuint32_t boxes[4] = {64, 1, 1, 1}, steps[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = cuuint64_t(size[slot[i]]);
    // a dimension of one is never stepped along: any valid stride serves
    strides[i] = size[slot[i]] > 1 ? cuuint64_t(stride[slot[i]]) * 2 : cuuint64_t(c.dim) * 2;
    if (strides[i] == 0) return false;
    if (slot[i] == 1) boxes[i + 1] = cuuint32_t(box);
  }
  return encode(map, c.dtype == DART_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace: error word (256 bytes), joints, then the parts.
constexpr size_t kJointBytes = (sizeof(Joint) * kCtas + 255) / 256 * 256;
int slot_rows(long long T, long long group) {
  const long long r = T * group;
  return int(r < kBlockRows ? (r < 1 ? 1 : r) : kBlockRows);
}

template <typename T, int DH>
cudaError_t launch(const AttendParams& P, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  const int smem = 2 * DH * kHalfTileBytes + kRingBytes + int(sizeof(Shared));
  cudaError_t e =
      settled(cudaFuncSetAttribute(attend_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (e != cudaSuccess) return e;
  // no more CTAs than run together: the spans are equal, so a CTA of a second round would double the time
  const int sms = device_sms(), ctas = sms > 0 && sms < kCtas ? sms : kCtas;
  e = launch_kernel(attend_kernel<T, DH>, ctas, kThreads, smem, s, P, km, vm);
  if (e != cudaSuccess) return e;
  // the join's CTAs take their places while the last attention CTAs finish, and wait there
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, (P.slot_rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(128 * DH);
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return settled(cudaLaunchKernelEx(&cfg, join_kernel<T, DH>, P));
}

}  // namespace
}  // namespace dart

extern "C" size_t dart_attention_workspace_bytes(int T, int B, int q_heads, int heads, int dim) {
  using namespace dart;
  if (T < 0 || B < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || dim < 8 || dim > 128 || dim % 8 != 0)
    return 0;
  const size_t cols = dim <= 64 ? 64 : 128;
  const size_t rows = slot_rows(T, q_heads / heads);
  return kCtrlBytes + kJointBytes + size_t(kCtas) * 2 * (cols / 4 * rows + (rows + 1) / 2) * sizeof(float4);
}

extern "C" int dart_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int q_heads,
                                   int T, int B, const int32_t* lengths, const int32_t* starts,
                                   const uint32_t* mask, int N, float scale, const dart_cache_t* cache,
                                   void* out, int64_t out_token_stride, int64_t out_head_stride, float* out_lse,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  using namespace dart;
  if (T < 0 || T > (1 << 26) || B < 0 || q_heads < 1 || q_heads > 65535 || N < 0 || N > kMaxN)
    return DART_ERR_INVALID_ARG;
  if ((long long)T * q_heads >= (1ll << 31)) return DART_ERR_INVALID_ARG;
  const int rc = check_cache(cache, B);
  if (rc) return rc;
  if (q_heads % cache->heads != 0 || !std::isfinite(scale * 1.44269504f)) return DART_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return DART_OK;
  if (cache->pages < 1 || cache->table_width < 1) return DART_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !mult8(q_token_stride, q_head_stride) ||
      !mult8(out_token_stride, out_head_stride) || !lengths || !starts || (N > 0 && !mask))
    return DART_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) != 0 ||
      workspace_bytes < dart_attention_workspace_bytes(T, B, q_heads, cache->heads, cache->dim))
    return DART_ERR_WORKSPACE;
  const dart_cache_t& c = *cache;
  AttendParams P;
  P.q = q; P.out = out; P.lse = out_lse;
  P.q_ts = q_token_stride; P.q_hs = q_head_stride;
  P.o_ts = out_token_stride; P.o_hs = out_head_stride;
  P.Hq = q_heads; P.Hkv = c.heads; P.G = q_heads / c.heads; P.D = c.dim;
  P.T = T; P.B = B; P.N = N; P.MW = (N + 31) / 32;
  P.lengths = lengths; P.starts = starts; P.mask = mask;
  // the least positive number for scale 0: any finite score becomes next to nothing, -inf stays -inf
  P.c = scale == 0.f ? std::numeric_limits<float>::denorm_min() : std::fabs(scale) * 1.44269504088896341f;
  P.negate = scale < 0.f ? 1u << 13 : 0u;
  P.wide_out = c.dim % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 31) == 0 &&
               ((out_token_stride | out_head_stride) & 15) == 0;
  P.table = c.table; P.table_stride = c.table_stride;
  P.cap = (long long)c.table_width * c.page;
  P.by_group = fast_div(uint32_t(P.G));
  P.by_page = fast_div(uint32_t(c.page));
  P.page = c.page; P.pages = c.pages; P.box = gcd(c.page, kTile);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.err = reinterpret_cast<uint32_t*>(ws);
  P.joints = reinterpret_cast<Joint*>(ws + kCtrlBytes);
  P.parts = reinterpret_cast<float4*>(ws + kCtrlBytes + kJointBytes);
  P.slot_rows = slot_rows(T, P.G);
  P.v = c.v; P.v_ps = c.v_page_stride; P.v_rs = c.v_row_stride; P.v_hs = c.v_head_stride;
  P.wait_limit = rows_wait_limit();
  CUtensorMap km, vm;
  if (!cache_map(c, c.k, c.k_page_stride, c.k_row_stride, c.k_head_stride, P.box, &km, P.k_slot) ||
      !cache_map(c, c.v, c.v_page_stride, c.v_row_stride, c.v_head_stride, P.box, &vm, P.v_slot))
    return DART_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c.dtype == DART_F16)
    e = c.dim <= 64 ? launch<__half, 1>(P, km, vm, s) : launch<__half, 2>(P, km, vm, s);
  else
    e = c.dim <= 64 ? launch<__nv_bfloat16, 1>(P, km, vm, s) : launch<__nv_bfloat16, 2>(P, km, vm, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
