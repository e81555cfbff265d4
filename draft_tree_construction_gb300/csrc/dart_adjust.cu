// dart_adjust.cu -- K5: penalties for repeated tokens, biases and grammar
// masks on logits, in one pass from the input rows to the output rows.
//
// Mathematics: x = z;  if counted: x = z (1 / r or r) - f cnt - p;  x += bias;
// -inf where the grammar bans the token; fp32, rounded once.
//
// What bounds it: memory, one read of the logits that are kept and one write of
// all.  What a row needs beyond its own elements is small and shared: how often
// each token occurs in the sequence's history, and the summed bias of each
// token.  So a CTA owns a slice of the vocabulary of one sequence, counts the
// history and sums the biases of that slice in shared memory once, and then
// copies that slice of its rows, whole vectors at a time, through a ring of
// shared-memory rows that cp.async fills ahead; a vector that the grammar bans is
// written without being read.  The few elements that are counted or biased are
// changed in the ring, each by a lane that keeps its change in registers from
// row to row.
//
// Measured (GB300, bf16, kernel alone):
//   64 x 8 rows of 151936, 2048 tokens of history, 300 biases   59 us, 5.3 TB/s
//   4 trees of 497 rows of 151936, 4096 tokens, one mask each  215 us, 5.3 TB/s
//   256 x 8 rows of 32000 (fp16), masks that keep 2% of a row   55 us: 2.6 TB/s
//     of what has to move, 4.3 TB/s of the 235 MB that do (131 written; 104 read,
//     since a kept logit brings its 128-byte line).  As long as with masks that
//     keep everything (56 us, 270 MB); 39 us with masks that keep nothing.  Its
//     1024 CTAs are 3.4 rounds: 228 sequences, three rounds, take 46 us
//   8 rows of 151936 of one sequence                            4.4 us
// Looking into every vector for touched elements instead took 99 and 359 us for
// the first two, registers in place of the ring 73 and 245 us, but 49 us for the
// masked rows.
#include <algorithm>
#include <cmath>

#include "dart_launch.h"

namespace dart {
namespace {

constexpr int kAdjThreads = 256;
constexpr int kAdjWarps = kAdjThreads / 32;
constexpr int kAdjVecs = 4;                                // 16-byte vectors a lane takes of a row
constexpr int kSparse = 24;                                // touched tokens of a block that are set one by one (8: 82
                                                           // for 77 us with 16384 tokens of history, 209 for 212 with 4096)
constexpr int kFix = kSparse * kAdjVecs / 32;              // ... and those of a warp's blocks, per lane
constexpr int kDepth = 3;                                  // rows under way per warp (2: 62 us for 58; 4 leave one CTA an SM: 80)
constexpr int kRingBytes = kDepth * kAdjWarps * kAdjVecs * 512;
constexpr int kMaxBias = 1024;                             // biases per sequence
constexpr int kCountBits = 21;                             // a token's count: history and path
constexpr int kMaxHistory = 1 << 20;
static_assert(kMaxHistory + kMaxN < (1 << kCountBits) && kMaxBias + 1 <= (1 << (32 - kCountBits)), "a place's word");
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

// Predicated loads that leave v alone otherwise, so that no register is copied
// (and nothing waits) between the load and the use.
__device__ __forceinline__ void ldg_word(uint32_t& v, const void* p, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.u32 %0, [%1];\n\t}"
               : "+r"(v) : "l"(p), "r"(uint32_t(on)) : "memory");
}
__device__ __forceinline__ void ldg_byte(uint32_t& v, const void* p, bool on) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.u8 %0, [%1];\n\t}"
               : "+r"(v) : "l"(p), "r"(uint32_t(on)) : "memory");
}
// One element's bits.
template <typename T>
__device__ __forceinline__ void ldg_elem(uint32_t& v, const T* p, bool on) {
  if (sizeof(T) == 4) {
    ldg_word(v, p, on);
  } else {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}"
                 : "+r"(v) : "l"(p), "r"(uint32_t(on)) : "memory");
  }
}
template <typename T>
__device__ __forceinline__ T elem_of(uint32_t v) {
  T x;
  memcpy(&x, &v, sizeof(T));
  return x;
}
// Logits pass through once: keep them out of the way of what is used again.
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

// The vector with -inf where the mask is 0.
template <typename T>
__device__ __forceinline__ uint4 ban(uint4 u, uint4 m) {
  constexpr uint32_t kInf = Elem<T>::kNegInf;
  return make_uint4((u.x & m.x) | (kInf & ~m.x), (u.y & m.y) | (kInf & ~m.y), (u.z & m.z) | (kInf & ~m.z),
                    (u.w & m.w) | (kInf & ~m.w));
}

// How the rows lie: every one begins on a 16-byte boundary, in and out; every
// one is as far from such a boundary in as it is out; or neither, and elements
// are taken one by one.  64 x 8 rows of 151936 with biases: 59 us aligned, 70 us
// shifted (an odd row length: a block of an unaligned row leaves a vector's worth
// of elements at its ends to be read and written singly), 330 us one by one (2
// bytes a lane and instruction).
enum Rows { kAligned, kShifted, kSingle };
template <typename T, int ROWS>
__global__ void __launch_bounds__(kAdjThreads, 2)
adjust_kernel(const AdjustParams P) {
  constexpr int E = 16 / int(sizeof(T));
  constexpr int kBlk = kBlock<T>, kCta = kSlice<T>, kWords = kCta / 32;
  constexpr uint32_t kAll = (1u << E) - 1u;
  constexpr bool kRing = ROWS != kSingle;
  // the ring: kDepth rows of each warp's vectors, on their way from memory or worked on
  extern __shared__ __align__(16) unsigned char smem[];
  // a place's word: 1 + its index in the bias list (0: not biased), and how often its token is counted
  uint32_t* counts = reinterpret_cast<uint32_t*>(smem + (kRing ? kRingBytes : 0));    // [kCta], with penalties or biases
  __shared__ uint32_t touched[kWords];             // place is counted or biased
  __shared__ uint32_t on_path[kWords];             // place's token is on the present row's path
  __shared__ int32_t list_id[kMaxBias];            // the slice's biases, in their order
  __shared__ float list_val[kMaxBias];             // ... the first entry of an id holding the id's sum
  __shared__ uint16_t list_own[kAdjWarps][32 * kFix];      // each warp's touched places in blocks that have few
  __shared__ uint32_t row_ok[kRing ? kDepth : 1][kAdjThreads];      // grammar bits of the rows in the ring
  __shared__ uint4 spread[1 << E];                 // the mask of a vector whose elements are the bits of the index
  __shared__ int16_t toks[kMaxN];                  // the places of the tree's tokens, -1 outside the slice
  __shared__ int32_t warp_n[kMaxBias / kAdjThreads][kAdjWarps];

  const int b = blockIdx.z, slice = blockIdx.x, slices = int(P.by_slices.d);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const dart_adjust_t& a = P.a;
  // token -> its place in the slice, -1 if it belongs to another or to none
  auto local = [&](int32_t token) {
    const int blk = token / kBlk, k = P.by_slices.div(blk);
    return uint32_t(token) < uint32_t(P.V) && blk - k * slices == slice ? k * kBlk + token % kBlk : -1;
  };

  // From here to the end a warp copies and changes its own blocks only: block i
  // lies at place (8 i + warp) * kBlk of the slice and holds the tokens from token(i) on.
  auto place = [&](int i) { return (kAdjWarps * i + warp) * kBlk; };
  auto token = [&](int i) { return ((kAdjWarps * i + warp) * slices + slice) * kBlk; };
  auto size = [&](int i) { return min(P.V - token(i), kBlk); };          // <= 0 behind the vocabulary
  const int r_begin = blockIdx.y * P.row_group, r_end = min(P.R, r_begin + P.row_group);
  const T* in = static_cast<const T*>(P.in) + ((long long)b * P.R + r_begin) * P.in_stride;
  T* out = static_cast<T*>(P.out) + ((long long)b * P.R + r_begin) * P.out_stride;
  const uint32_t* allow =
      a.allowed ? a.allowed + (long long)b * a.allowed_seq_stride + (long long)r_begin * a.allowed_row_stride : nullptr;

  // The ring: a lane's vectors lie `step` tokens apart, from v0 + head on, where
  // `head` elements come before the first 16-byte boundary of each block of the
  // row (0 for aligned rows; blocks are multiples of 16 bytes).  Rows are copied
  // there kDepth - 1 rows ahead (but for vectors that the grammar bans), changed
  // there, and written from there with the banned elements replaced.
  const int step = kAdjWarps * slices * kBlk, v0 = token(0) + lane * E;
  constexpr int kPlaceStep = kAdjWarps * kBlk, kRowBytes = kAdjWarps * kAdjVecs * 512;
  unsigned char* ring = smem + warp * (kAdjVecs * 512);            // + slot * kRowBytes
  auto row_of = [&](int r) { return in + (long long)(r - r_begin) * P.in_stride; };
  auto head_of = [&](int r) {
    return ROWS == kAligned
               ? 0
               : int((16u - unsigned(reinterpret_cast<uintptr_t>(row_of(r)) & 15u)) & 15u) / int(sizeof(T));
  };
  auto whole = [&](int i, int head) { return head + (lane + 1) * E <= size(i); };
  // grammar bits: asked for a row before the row's copy begins (a vector's bits
  // lie in one byte, or in two if the rows are shifted)
  uint32_t bits[kAdjVecs], more_bits[kAdjVecs];
#pragma unroll
  for (int i = 0; i < kAdjVecs; ++i) bits[i] = more_bits[i] = kFull;
  const int mask_bytes = ((P.V + 31) >> 5) * 4;
  auto ask = [&](int r) {
    const uint8_t* src = reinterpret_cast<const uint8_t*>(allow + (long long)(r - r_begin) * a.allowed_row_stride);
    const int head = head_of(r), at = (v0 + head) >> 3;
#pragma unroll
    for (int i = 0; i < kAdjVecs; ++i) {
      const bool on = r < r_end && whole(i, head);
      ldg_byte(bits[i], src + at + i * (step / 8), on);
      if (ROWS == kShifted)
        ldg_byte(more_bits[i], src + at + i * (step / 8) + 1, on && at + i * (step / 8) + 1 < mask_bytes);
    }
  };
  auto copy = [&](int r, int slot) {
    uint32_t ok = 0u;
    const int head = head_of(r);
    const T* src = row_of(r) + v0 + head;
#pragma unroll
    for (int i = 0; i < kAdjVecs; ++i) {
      const uint32_t two = ROWS == kShifted ? (bits[i] & 0xFFu) | (more_bits[i] << 8) : bits[i];
      const uint32_t k = (two >> ((v0 + head) & 7)) & kAll;
      ok |= k << (8 * i);
      cp_async16(ring + slot * kRowBytes + i * 512 + lane * 16, src + i * step, r < r_end && whole(i, head) && k != 0u);
    }
    cp_async_commit();
    row_ok[slot][tid] = ok;
    if (allow) ask(r + 1);
  };

  // Everything that the slice needs from memory is asked for before anything waits
  // (of a long history the first kAhead entries a thread, then kMore at a time).
  if (kRing && allow) ask(r_begin);
  constexpr int kAhead = 8, kMore = 16, kBiasAhead = kMaxBias / kAdjThreads;
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
  const bool touching = P.count || a.bias_count > 0, paths = P.count && a.N > 0;

  if constexpr (kRing) {
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) copy(r_begin + k, k);
  }

  for (int i = tid; i < kWords; i += kAdjThreads) touched[i] = on_path[i] = 0u;
  if (touching)
    for (int i = tid; i < kCta / 4; i += kAdjThreads) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
  for (int i = tid; i < (1 << E); i += kAdjThreads) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = E == 4 ? 0u - ((uint32_t(i) >> j) & 1u)
                    : ((i >> (2 * j)) & 1 ? 0xFFFFu : 0u) | ((i >> (2 * j)) & 2 ? 0xFFFF0000u : 0u);
    spread[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (paths)
    for (int i = tid; i < a.N; i += kAdjThreads) toks[i] = int16_t(local(a.tokens[(long long)b * a.N + i]));
  __syncthreads();
  auto tally = [&](int i, int32_t token) {
    const int t = i < len ? local(token) : -1;
    if (t >= 0) {
      atomicAdd(&counts[t], 1u);
      atomicOr(&touched[t >> 5], 1u << (t & 31));
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) tally(tid + k * kAdjThreads, id[k]);
  for (int i0 = tid + kAhead * kAdjThreads; i0 < len; i0 += kMore * kAdjThreads) {
    int32_t more[kMore];
#pragma unroll
    for (int k = 0; k < kMore; ++k) more[k] = i0 + k * kAdjThreads < len ? hist[i0 + k * kAdjThreads] : -1;
#pragma unroll
    for (int k = 0; k < kMore; ++k) tally(i0 + k * kAdjThreads, more[k]);
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
      list_val[i] = s;                           // no other entry reads it: only the first of an id reads values
      atomicAdd(&counts[t], uint32_t(i + 1) << kCountBits);
      atomicOr(&touched[t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();

  if (token(0) >= P.V) return;
  const int MW = (a.N + 31) >> 5;

  // The touched places of blocks that have few of them go to a list, a lane
  // taking every 32nd; the other blocks (bits of `dense`) look for theirs vector by vector.
  int own = 0;
  uint32_t dense = 0u;
  {
    constexpr int kPer = kBlk / 32;              // words per block
    uint32_t m = lane < kAdjVecs * kPer ? touched[place(lane / kPer) / 32 + lane % kPer] : 0u;
    int n = __popc(m), in_block = n;
#pragma unroll
    for (int o = 1; o < kPer; o <<= 1) in_block += __shfl_xor_sync(kFull, in_block, o);
    const bool many = in_block > kSparse;
#pragma unroll
    for (int i = 0; i < kAdjVecs; ++i) dense |= uint32_t(__shfl_sync(kFull, int(many), i * kPer)) << i;
    if (many) m = 0u, n = 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    own = __shfl_sync(kFull, incl, 31);
    for (int at = incl - n; m; m &= m - 1, ++at)
      list_own[warp][at] = uint16_t(place(lane / kPer) + 32 * (lane % kPer) + __ffs(m) - 1);
    __syncwarp();
  }
  // a touched element: scaled if counted, then what it gains, rounded once in fp32
  struct Change { int v; bool counted; float gain; };
  auto change = [&](int t) {
    const uint32_t word = counts[t], c = word & ((1u << kCountBits) - 1u), i = word >> kCountBits;
    const float bias = i ? list_val[i - 1] : 0.f;
    Change h;
    h.v = ((t / kBlk) * slices + slice) * kBlk + t % kBlk;
    h.counted = c != 0u;
    h.gain = c ? bias - fmaf(freq, float(c), pres) : bias;
    return h;
  };
  auto apply = [&](T raw, const Change& h) {
    const float x = Elem<T>::get(raw);
    return Elem<T>::put(fmaf(x, h.counted ? (x > 0.f ? inv_rep : rep) : 1.f, h.gain));
  };
  auto keeps = [](const uint32_t* allow, int v) { return !allow || ((allow[v >> 5] >> (v & 31)) & 1u); };
  auto marked = [&](int t) { return (on_path[t >> 5] >> (t & 31)) & 1u; };
  // this lane's touched elements stay in registers
  Change fix[kFix];
  int fix_at[kFix];
#pragma unroll
  for (int k = 0; k < kFix; ++k) {
    fix_at[k] = lane + 32 * k < own ? list_own[warp][lane + 32 * k] : -1;
    fix[k].v = 0;
    if (fix_at[k] >= 0) fix[k] = change(fix_at[k]);
  }

  // the nodes whose tokens this warp owns, 32 nodes a lane
  uint32_t own_nodes = 0u;
  if (paths)
    for (int k = 0; k < 32 && 32 * lane + k < a.N; ++k) {
      const int t = toks[32 * lane + k];
      own_nodes |= uint32_t(t >= 0 && t / kBlk % kAdjWarps == warp) << k;
    }
  auto node_bits = [&](int r) {       // this lane's word of row r's path, the warp's own nodes
    const int node = r - (P.R - a.N);
    return paths && r < r_end && node >= 0 && lane < MW ? a.mask[((long long)b * a.N + node) * MW + lane] & own_nodes
                                                         : 0u;
  };
  auto each = [&](uint32_t path, auto&& f) {
    for (uint32_t m = path; m; m &= m - 1) f(int(toks[32 * lane + __ffs(m) - 1]));
    __syncwarp();
  };
  // The tokens of a row's path join the counts and are marked, for the time of the row.
  auto path_in = [&](uint32_t path) {
    each(path, [&](int t) {
      atomicAdd(&counts[t], 1u);
      atomicOr(&on_path[t >> 5], 1u << (t & 31));
    });
  };
  auto path_out = [&](uint32_t path) {
    __syncwarp();
    each(path, [&](int t) {
      atomicAnd(&on_path[t >> 5], ~(1u << (t & 31)));
      atomicSub(&counts[t], 1u);
    });
  };
  // one element by itself: token v, at place t
  auto single = [&](T raw, bool keep, int t) {
    T y = Elem<T>::put(-INFINITY);
    if (keep) y = touching && counts[t] ? apply(raw, change(t)) : raw;
    return y;
  };

  if constexpr (kRing) {
    // the touched elements of a dense block's vector, at place t
    auto dense_set = [&](Vec<T>& x, uint32_t hit, int t) {
      uint32_t c[E];
      if constexpr (ROWS == kAligned) {
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<uint4*>(c + e) = *reinterpret_cast<const uint4*>(counts + t + e);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) c[e] = counts[t + e];
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t n = c[e] & ((1u << kCountBits) - 1u), i = c[e] >> kCountBits;
        float gain = i ? list_val[i - 1] : 0.f;
        if (n) gain -= fmaf(freq, float(n), pres);
        const float y = Elem<T>::get(x.e[e]);
        const T z = Elem<T>::put(fmaf(y, n ? (y > 0.f ? inv_rep : rep) : 1.f, gain));
        if ((hit >> e) & 1u) x.e[e] = z;
      }
    };
    // A block's elements before its first and behind its last whole vector are
    // set singly: lane E i + s takes the s-th of block i (and the s + E-th, which
    // only the vocabulary's last block can have).
    const int tail_blk = lane / E, tail_s = lane % E;
    const int tail_n = tail_blk < kAdjVecs ? max(size(tail_blk), 0) : 0;
    auto tail_at = [&](int head, int s) {       // its offset in the block, -1 if there is none
      const int vecs = max(tail_n - head, 0) / E * E;
      return s < tail_n - vecs ? (s < head ? s : vecs + s) : -1;
    };
    const bool tails = __any_sync(kFull, ROWS == kShifted || tail_at(0, tail_s) >= 0);
    uint32_t tail_raw = 0u, tail_word = kFull;
    auto tail_read = [&](int r) {
      const int k = tails && r < r_end ? tail_at(head_of(r), tail_s) : -1;
      const int v = token(tail_blk) + k;
      ldg_elem(tail_raw, row_of(r) + v, k >= 0);
      ldg_word(tail_word, allow + (long long)(r - r_begin) * a.allowed_row_stride + (v >> 5), k >= 0 && allow);
    };
    tail_read(r_begin);

    uint32_t path = node_bits(r_begin);
    int slot = 0;
    for (int r = r_begin; r < r_end; ++r) {
      copy(r + kDepth - 1, slot == 0 ? kDepth - 1 : slot - 1);
      const uint32_t next_path = node_bits(r + 1);
      const int head = head_of(r);
      // where the element at place t lies in the warp's part of the row, nullptr if it is set singly
      auto element = [&](int t) -> T* {
        const int i = t / kPlaceStep, k = t % kBlk - head;
        if (ROWS == kShifted && unsigned(k) >= unsigned(max(size(i) - head, 0) / E * E)) return nullptr;
        return reinterpret_cast<T*>(ring + slot * kRowBytes + i * 512) + k;
      };
      cp_async_wait<kDepth - 1>();
      __syncwarp();
      const bool walked = paths && __any_sync(kFull, path != 0u);
      if (walked) path_in(path);
      if (own > 0) {
#pragma unroll
        for (int k = 0; k < kFix; ++k)
          if (32 * k < own && fix_at[k] >= 0 && !(walked && marked(fix_at[k]))) {
            T* e = element(fix_at[k]);
            if (e) *e = apply(*e, fix[k]);
          }
      }
      const T tail_was = elem_of<T>(tail_raw);
      const uint32_t tail_kept = tail_word;
      if (walked) {
        __syncwarp();
        each(path, [&](int t) {               // the lane that clears the mark sets the element
          const uint32_t bit = 1u << (t & 31);
          if ((on_path[t >> 5] & bit) && !((dense >> (t / kPlaceStep)) & 1u) &&
              (atomicAnd(&on_path[t >> 5], ~bit) & bit)) {
            T* e = element(t);
            if (e) *e = apply(*e, change(t));
          }
        });
      }
      __syncwarp();
      const uint32_t ok = row_ok[slot][tid];
      T* dst = out + v0 + head;
#pragma unroll
      for (int i = 0; i < kAdjVecs; ++i) {
        Vec<T> x;
        x.u = *reinterpret_cast<const uint4*>(ring + slot * kRowBytes + i * 512 + lane * 16);
        const uint32_t k = (ok >> (8 * i)) & kAll;
        const bool on = whole(i, head);
        if ((dense >> i) & 1u) {
          const int t = place(i) + head + lane * E;
          uint32_t hit = 0u;
          if (on) {
            hit = bits_at(touched, t, kWords);
            if (walked) hit |= bits_at(on_path, t, kWords);
            hit &= k;
          }
          if (hit) dense_set(x, hit, t);
        }
        if (allow) x.u = ban<T>(x.u, spread[k]);
        if (on) stg_stream(dst + i * step, x.u);
      }
      if (tails) {
        const int k = tail_at(head, tail_s);
        if (k >= 0) {
          const int v = token(tail_blk) + k;
          out[v] = single(tail_was, (tail_kept >> (v & 31)) & 1u, place(tail_blk) + k);
        }
        const int far = tail_at(head, tail_s + E);
        if (far >= 0 && tail_blk < kAdjVecs) {
          const int v = token(tail_blk) + far;
          out[v] = single(row_of(r)[v], keeps(allow ? allow + (long long)(r - r_begin) * a.allowed_row_stride : nullptr, v),
                          place(tail_blk) + far);
        }
        tail_read(r + 1);
      }
      if (walked) path_out(path);
      out += P.out_stride;
      path = next_path;
      slot = slot + 1 < kDepth ? slot + 1 : 0;
    }
    cp_async_wait<0>();
  } else {
    for (int r = r_begin; r < r_end; ++r) {
      const uint32_t path = node_bits(r);
      const bool walked = paths && __any_sync(kFull, path != 0u);
      if (walked) path_in(path);
#pragma unroll 1
      for (int i = 0; i < kAdjVecs; ++i)
#pragma unroll 4
        for (int k = lane; k < size(i); k += 32) {
          const int v = token(i) + k;
          out[v] = single(in[v], keeps(allow, v), place(i) + k);
        }
      if (walked) path_out(path);
      in += P.in_stride;
      out += P.out_stride;
      if (allow) allow += a.allowed_row_stride;
    }
  }
}

template <typename T, int ROWS>
cudaError_t launch_rows_as(const AdjustParams& P, dim3 grid, cudaStream_t stream) {
  constexpr int kMost = 4 * kSlice<T> + (ROWS != kSingle ? kRingBytes : 0);
  const cudaError_t e =
      settled(cudaFuncSetAttribute(adjust_kernel<T, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost));
  if (e != cudaSuccess) return e;
  const bool touching = P.count || P.a.bias_count > 0;
  return launch_kernel(adjust_kernel<T, ROWS>, grid, kAdjThreads, kMost - (touching ? 0 : 4 * kSlice<T>), stream, P);
}

template <typename T>
cudaError_t launch_adjust(AdjustParams P, int B, cudaStream_t stream) {
  const int slices = (P.V + kSlice<T> - 1) / kSlice<T>;
  P.by_slices = fast_div(uint32_t(slices));
  // Rows per CTA.  304 CTAs run together; each begins and counts, for as long as `count`
  // rows take, before its first row, and one that began late or holds the crowded ids
  // ends up to 0.4 of its rows after the others.  So w rounds of CTAs, each with a share
  // of the rows, take about w (count + rows) + 0.4 rows, and the least of that is taken:
  //   4 trees of 497 rows of 151936, 4096 tokens: 232, 218, 216, 220, 224 us with w = 1..5
  //   6 trees of 285 rows of 13938, 511 tokens: 42, 35, 38, 42 us with w = 1..4
  //   64 x 8 rows of 151936, 2048 tokens: 59 and 68 us with w = 4 and 8
  //   24 x 5 fp32 rows of 32000, 14312 tokens: 20 and 42 us with w = 1 and 4
  //   178 trees of 286 rows of 9353, 583 tokens: 912, 863, 805 us with w = 4, 5 and 6
  const long long per = (long long)slices * B, together = 152 * 2;
  const float count = 2.f + (P.count ? float(P.a.history_width) / 1600.f : 0.f);
  long long groups = 1;
  float least = 3e38f;
  for (int w = 1; w <= 16; ++w) {
    long long g = std::max(1ll, std::min(w * together / per, (long long)P.R));
    const long long rows = (P.R + g - 1) / g;
    g = (P.R + rows - 1) / rows;
    const float cost = float((per * g + together - 1) / together) * (count + float(rows)) + 0.4f * float(rows);
    if (cost < least) least = cost, groups = g;
    if (g == P.R) break;
  }
  if (groups > 65535) groups = 65535;
  P.row_group = int((P.R + groups - 1) / groups);
  const dim3 grid(slices, (P.R + P.row_group - 1) / P.row_group, B);
  const uintptr_t in = reinterpret_cast<uintptr_t>(P.in), out = reinterpret_cast<uintptr_t>(P.out);
  const uintptr_t in_step = uintptr_t(P.in_stride) * sizeof(T), out_step = uintptr_t(P.out_stride) * sizeof(T);
  if (((in | out | in_step | out_step) & 15) == 0) return launch_rows_as<T, kAligned>(P, grid, stream);
  if ((((in ^ out) | (in_step ^ out_step)) & 15) == 0) return launch_rows_as<T, kShifted>(P, grid, stream);
  return launch_rows_as<T, kSingle>(P, grid, stream);
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
  if (a.history_width < 0 || a.history_width > kMaxHistory || a.bias_count < 0 || a.bias_count > kMaxBias || a.N < 0 || a.N > kMaxN)
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
