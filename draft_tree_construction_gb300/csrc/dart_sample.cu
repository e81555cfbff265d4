// dart_sample.cu -- K12: tokens drawn from logits with temperature, top-k, top-p and
// min-p, one given random number a row.
//
// Mathematics.  With the row's tokens in descending order of their logits (lower id
// first where they are equal) and w_i = e^((z_i - max) / T), a prefix of that order is
// kept: n = max(1, min(k, n_p, n_m)), n_p the first place where the running sum reaches
// p times the sum of the first k, n_m the number of w_i >= min_p.  The token is the
// first whose running sum exceeds u times the sum of the n kept ones.
//
// Rows are not sorted.  What matters of a row is a few hundred tokens near its largest
// logit, so one reading finds the largest, a second one (from L2) lists the tokens within
// 2^-12 of its weight and sums the others' weights, and the list alone is sorted and
// summed.  Where a limit or the random number reaches further down, a histogram of the
// distances from the largest (1/64 of a binary order each) says how far, and the second
// reading is repeated: to that depth, or, where more than 2048 tokens lie before it, for
// the tokens around that place alone, those before it only summed.  What is left (many
// equal values, several limits far down) goes by general(), a histogram of the values.
//
// Which token a random number falls on is a matter of the last bits of sums over the
// whole vocabulary, so weights are 64-bit integers, good to 2^-42 of themselves (to 2^-28
// below 2^-16 of the largest) and to a part, and their sums exact in any order.  Only sums of
// what is not listed are taken with less (the bounds are at Tail and Mid); where a place lies
// so near to an edge that this could matter, the next form decides, general() at last.  A
// call gives the same bits every time.
//
// Rows that are fewer than the SMs are shared by up to eight CTAs of a cluster, which hand
// their largest logit, list and sum to the first one through distributed shared memory.
//
// Measured (GB300, graph-replayed; the floor is one reading at the copy rate):
//   one row of 151936 bf16, top-k and top-p      15..21 us (90 where it goes by general()): three
//     cluster barriers, two readings, the list
//   4 x 497 rows of 151936 bf16, all limits      126..349 us, floor 90; 115 where all rows are greedy
//   64 x 79 rows of 32000 fp16, top-p 0.7..0.99  311..457 us, floor 48: half of it in the tenth of the
//     rows whose sums reach far down (an integer add in shared memory takes 16 cycles a warp); 77 where
//     all are greedy, 120 with min-p alone
//   500 rows of 32000 fp32, temperature alone    89..155 us, floor 9.6: two rounds of rows, as long as their
//     longest; 29 with min-p alone
#include "dart_launch.h"

namespace dart {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kThreads = 512;                // of general(), and of a row that is shared
constexpr int kManyThreads = 256, kManyCtas = 4;   // of one row of many
constexpr int kParts = 2048;                 // of a bin that is divided again

struct SampleParams {
  const void* logits;
  long long stride;
  const float *uniforms, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tokens;
  float* probs;
  int R, V, shift;                           // a weight of 1 is 2^shift
  int ranks;                                 // CTAs that share a row
  long long rows;
};

// Which 16-bit magnitudes have bins of their own: kLow .. kHigh - 1.  bf16: 2^-8 .. 2^9;
// f16: 2^-3 .. 2^6; f32 goes by its upper half, as bf16.
template <typename T> struct Fine { static constexpr int kLow = 119 << 7, kHigh = 136 << 7, kInf = 0x7F80; };
template <> struct Fine<__half> { static constexpr int kLow = 12 << 10, kHigh = 21 << 10, kInf = 0x7C00; };

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
  // The distance to the next logit of the same exponent, of 16-bit ones with normal magnitudes.
  static __device__ __forceinline__ int exponent(uint32_t bits) { return int(bits) >> (F::kInf == 0x7C00 ? 10 : 7); }   // and sign
  static __device__ __forceinline__ float step(uint32_t bits) {
    const int e = exponent(bits & 0x7FFFu);
    return __uint_as_float(uint32_t(F::kInf == 0x7C00 ? e - 25 + 127 : e - 7) << 23);
  }
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
// Two forms, the top and the factor c = log2(e) / T in two parts for both; `table` has
// 2^-j/256 in units of 2^-63, `shift` says that 1 is 2^shift.
struct Mid {                                 // 2^-y to 2^-28 of itself, less a part
  float top, c_hi, c_lo;
  int shift;
  const uint64_t* table;
  // y = (top - z) c: the difference exactly in two parts, the product in two
  __device__ __forceinline__ float distance(float z, float& rest) const {
    const float d = top - z, v = d - top, e = (top - (d - v)) - (z + v), y = d * c_hi;
    rest = fmaf(d, c_hi, -y) + fmaf(d, c_lo, e * c_hi);
    return y;
  }
  // y = whole + j / 256 + r, |r| <= 2^-9: 2^-r - 1 in fp32 (half a unit of 2^-31), rounded to such
  // units (half of one), 2^-j/256 and the product cut to them (one each): 3 units of at least
  // 2^30 (1 - 2^-9), less than 2^-28 (2^-28.9 is the most that was seen)
  __device__ __forceinline__ uint64_t power(float y, float rest) const {
    constexpr float kRound = 12582912.f;     // 1.5 2^23: a sum with it is a whole number
    const float n = fmaf(y, 256.f, kRound);
    const int steps = __float_as_int(n) - __float_as_int(kRound);
    const float r = fmaf(n - kRound, -0.00390625f, y) + rest;
    const float s = r * fmaf(r, fmaf(r, -0.05550410866f, 0.2402265070f), -0.6931471806f);     // 2^-r - 1
    const int q = __float_as_int(fmaf(s, 2147483648.f, kRound)) - __float_as_int(kRound);
    const int a = int(uint32_t(table[steps & 255] >> 32));
    const uint32_t w = uint32_t(a) + uint32_t(int((long long)a * q >> 31));
    return (uint64_t(w) << (shift - 31)) >> (steps >> 8);
  }
  __device__ __forceinline__ uint64_t operator()(float z) const {
    float rest;
    const float y = distance(z, rest);
    return y < 62.f ? power(y, rest) : 0ull;
  }
};
struct Weigh : Mid {                         // to 2^-42 of itself, below 2^-16 as Mid
  // 2^-(y + rest) in units of 2^-63, 0 <= y < 62.  Where its terms are cut costs 2^-46.5 of itself,
  // y's own error, 2^-47 y ln 2 by the factor in two parts, 2^-43.5 at y = 16
  __device__ __forceinline__ uint64_t exact(float y, float rest) const {
    // y in units of 2^-48: whole part, 256ths, remainder r
    const long long Y = (long long)(y * 281474976710656.f) + __float2ll_rn(rest * 281474976710656.f);
    if (Y <= 0) return 1ull << 63;
    const int whole = int(Y >> 48), j = int(Y >> 40) & 255;
    // 2^-r = 1 - (x - x^2/2 + x^3/6 - x^4/24), x = r ln 2 < 2^-8, in units of 2^-64; the
    // powers need their upper 32 bits
    const uint64_t x = __umul64hi(uint64_t(Y & ((1ll << 40) - 1)) << 16, 0xb17217f7d1cf79abull);
    const uint32_t a = uint32_t(x >> 24);                              // units of 2^-40
    const uint64_t x2 = (uint64_t(a) * a) >> 17;                       // x^2 / 2
    const uint64_t x3 = (uint64_t(uint32_t(x2 >> 16)) * a) >> 24;      // x^3 / 2
    const uint64_t x4 = (uint64_t(uint32_t(x3 >> 8)) * a) >> 32;       // x^4 / 2
    // a third and a twelfth by 32-bit products, to 2^-47
    const uint64_t s = x - x2 + (uint64_t(__umulhi(uint32_t(x3 >> 16), 0x55555556u)) << 16) -
                       (uint64_t(__umulhi(uint32_t(x4 >> 8), 0x15555556u)) << 8);
    const uint64_t t = table[j];
    return (t - __umul64hi(t, s)) >> whole;
  }
  __device__ __forceinline__ uint64_t rounded(uint64_t w) const { return (w + (1ull << (62 - shift))) >> (63 - shift); }
  __device__ __forceinline__ uint64_t operator()(float z) const {
    if (z == top) return 1ull << shift;
    float rest;
    const float y = distance(z, rest);
    if (!(y < 62.f)) return 0ull;            // also top = +inf
    return y < 16.f ? rounded(exact(y, rest)) : power(y, rest);
  }
  // In units of 2^-63, and the factor from one logit to the next one `step` below, in 2^-64.
  __device__ __forceinline__ uint64_t fine(float z) const {
    float rest;
    const float y = distance(z, rest);
    return z == top ? 1ull << 63 : y < 62.f ? exact(y, rest) : 0ull;
  }
  __device__ __forceinline__ uint64_t ratio(float step) const {
    const float y = step * c_hi;
    if (!(y < 62.f)) return 0ull;
    const uint64_t w = exact(y, fmaf(step, c_hi, -y) + step * c_lo);
    return w >> 63 ? ~0ull : w << 1;
  }
};

// ---------------------------------------------------------------- the row
// The part of a row that a CTA reads: vectors v0 .. v1 of the aligned middle, and the
// elements before it (by the first CTA) and behind it (by the last).
template <typename T>
struct Slice {
  static constexpr int kPer = 16 / int(sizeof(T));
  const T* row;
  const uint4* body;
  int head, tail, V, v0, v1;
  bool first, last;
  __device__ __forceinline__ Slice(const T* r, int n, int rank, int ranks) : row(r), V(n) {
    head = min(n, int((16 - (reinterpret_cast<uintptr_t>(r) & 15)) & 15) / int(sizeof(T)));
    const int vecs = (n - head) / kPer, per = (vecs + ranks - 1) / ranks;
    tail = head + vecs * kPer;
    body = reinterpret_cast<const uint4*>(r + head);
    v0 = min(rank * per, vecs);
    v1 = min(v0 + per, vecs);
    first = rank == 0;
    last = rank == ranks - 1;
  }
  // All threads; one(i) of the single elements, vec(x, i) of the vectors, i the place of the (first) element.
  template <int NT, typename F, typename G>
  __device__ __forceinline__ void each(F&& one, G&& vec) const {
    constexpr int kUnroll = 4;
    const int t = threadIdx.x;
    if (first && t < head) one(t);
    if (last && tail + t < V) one(tail + t);
    for (int v = v0 + t; v < v1; v += NT * kUnroll) {
      uint4 x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v + u * NT < v1) x[u] = __ldg(body + v + u * NT);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (v + u * NT < v1) vec(x[u], head + (v + u * NT) * kPer);
    }
  }
};
// The upper 16 bits and the value of element k of a vector, or of a single one.
template <typename T>
__device__ __forceinline__ uint32_t bits_of(const uint4& x, int k) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 2) return k & 1 ? w[k >> 1] >> 16 : w[k >> 1] & 0xFFFFu;
  else return w[k] >> 16;
}
template <typename T>
__device__ __forceinline__ float value_of(const uint4& x, int k) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (sizeof(T) == 2) return to_float<T>(bits_of<T>(x, k));
  else return __uint_as_float(w[k]);
}
template <typename T> __device__ __forceinline__ float value_at(const T* row, int i) { return float(row[i]); }
template <typename T> __device__ __forceinline__ uint32_t bits_at(const T* row, int i) {
  if constexpr (sizeof(T) == 2) return reinterpret_cast<const uint16_t*>(row)[i];
  else return reinterpret_cast<const uint32_t*>(row)[i] >> 16;
}
// f(upper bits, value, place) of every logit of the slice that counts (not NaN, not -inf), in any order.
template <int NT, typename T, typename F>
__device__ __forceinline__ void each_logit(const Slice<T>& s, F&& f) {
  auto one = [&](uint32_t bits, float z, int i) {
    if (z > -INFINITY) f(bits, z, i);
  };
  s.template each<NT>([&](int i) { one(bits_at(s.row, i), value_at(s.row, i), i); },
         [&](const uint4& x, int i) {
#pragma unroll
           for (int k = 0; k < Slice<T>::kPer; ++k) one(bits_of<T>(x, k), value_of<T>(x, k), i + k);
         });
}

struct Place {                               // of a token in the order
  uint32_t key;                              // its logit
  uint32_t r;                                // tokens of that logit before it
  uint32_t count;                            // tokens of larger logits
  uint64_t weight;                           // their weight
};

constexpr int kList = 2048;                  // tokens that are listed
constexpr int kMaxRanks = 8;
enum Verdict : uint32_t { kDone, kPlan, kRefine, kRead, kGeneral };

struct Shared {
  uint64_t table[256];
  uint64_t warp_weight[32];
  uint64_t tails[kMaxRanks], heads[kMaxRanks];   // by rank, with the first CTA: the sums of what is not listed
  uint64_t at_weight, end_weight;            // what a search found
  uint32_t warp_count[32];
  uint64_t tops[kMaxRanks];                  // by rank, with every CTA: the largest logit, and what its part of top_k reaches
  uint32_t at_count, at_bin, end_count, at_end;
  uint32_t mine, others;                     // tokens listed by this CTA, and handed over to it
  uint32_t first;                            // greedy: the first place of the largest logit
  uint32_t verdict;
  float cut, cut_above;                      // tokens from cut up to below cut_above are listed
  float from, scale;                         // a plan's first distance, and its steps a binary order
  float least;                               // the smallest logit that min-p keeps
  float want, behind;                        // how far a plan has to reach: the weight up to there and behind it
};
// With the list: two arrays of kList words (tokens; running sums, or what the others hand over, or the plan's counts).
// In general(): the parts of a bin, then the bins.
struct Parts {
  uint64_t weight[kParts];
  uint32_t count[kParts];
};

// Exclusive sums over the CTA's threads, and the totals.
template <int NT>
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
  for (int i = 0; i < NT / 32; ++i) {
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

// sum times f, rounded down or up: f's 24 bits times 64; nothing for f <= 0 and NaN, sum from 1 on.
__device__ __forceinline__ uint64_t share_of(uint64_t sum, float f, bool up) {
  if (!(f > 0.f)) return 0ull;
  if (f >= 1.f) return sum;
  const uint32_t bits = __float_as_uint(f), m = (bits & 0x7FFFFFu) | 0x800000u, down = 150 - (bits >> 23);
  if ((bits >> 23) == 0 || down >= 128) return up ? 1ull : 0ull;
  const uint64_t lo = sum * m, hi = __umul64hi(sum, m);
  const uint64_t x = down < 64 ? (hi << (64 - down)) | (lo >> down) : hi >> (down - 64);
  const uint64_t rest = down < 64 ? lo & ((1ull << down) - 1) : lo | (hi & ((1ull << (down - 64)) - 1));
  return x + (up && rest ? 1ull : 0ull);
}

// w / sum, rounded once (to 2^-40 before that): both in two floats, one step of division.
__device__ __forceinline__ float ratio(uint64_t w, uint64_t sum) {
  const float a = __ull2float_rz(w), c = __ull2float_rz(sum);
  const float b = __ull2float_rn(w - uint64_t(a)), d = __ull2float_rn(sum - uint64_t(c));
  const float q = a / c, r = fmaf(-q, c, a) + fmaf(-q, d, b);
  return q + r / c;
}

struct Settings {
  float heat, top_p, min_p, u;
  int top_k;
  bool by_k, by_p, by_m;                     // limits that are set; by_k: below the vocabulary
  bool tail;                                 // the weight of what is not listed counts
  float least;                               // by_m: the smallest logit that it keeps
};

// A row's draw by the histogram of its values.  The order is by value, so counts and
// weights of values answer every question of place.  A 16-bit logit is its own bin where
// its magnitude is usual (the rest share three bins), and a bin's weight is its count
// times the weight of its one value.  Bins of several values (all of them where logits
// have 32 bits) have their weights summed element by element, and the one that a place
// falls into is divided again, 2048 parts at a time, until its parts hold one value each.
// Integer adds in shared memory bound it, one for each logit.
template <typename T>
__device__ __noinline__ void general(const SampleParams& P, const T* logits, long long at, const Weigh& weigh,
                                     const Settings& S, Shared* sh, unsigned char* scratch) {
  using B = Bins<T>;
  constexpr int kPer = (B::kCount + kThreads - 1) / kThreads;       // bins of a thread
  static_assert(kPer <= 64, "a warp looks at a thread's bins in two steps");
  Parts* parts = reinterpret_cast<Parts*>(scratch);
  uint64_t* bin_weight = reinterpret_cast<uint64_t*>(parts + 1);    // of bins of several values: all, or three
  uint32_t* bin_count = reinterpret_cast<uint32_t*>(bin_weight + (B::kSingle ? 4 : B::kCount + 1));
  auto slot = [](int bin) { return B::kSingle ? (bin == 0 ? 0 : bin == B::kMiddle ? 1 : 2) : bin; };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = P.V;
  const Slice<T> row(logits, V, 0, 1);

  // ---- counts of all bins
  __syncthreads();
  for (int i = tid; i < B::kCount; i += kThreads) bin_count[i] = 0;
  for (int i = tid; i < (B::kSingle ? 4 : B::kCount); i += kThreads) bin_weight[i] = 0;
  __syncthreads();
  // 16-bit logits of the three shared bins are set aside, where there are few of them
  uint16_t* aside = reinterpret_cast<uint16_t*>(parts->weight);
  constexpr uint32_t kAside = sizeof(parts->weight) / 2;
  if (tid == 0) sh->mine = 0;
  __syncthreads();
  // the bin by integers alone; -inf and NaN, whose magnitudes are the largest, are left out
  auto count = [&](uint32_t bits) {          // true: a shared bin's logit
    const int magnitude = int(bits & 0x7FFFu), d = min(max(magnitude, B::F::kLow - 1), B::F::kHigh) - (B::F::kLow - 1);
    if (magnitude >= B::F::kInf && bits != uint32_t(B::F::kInf)) return false;
    atomicAdd(&bin_count[bits & 0x8000u ? B::kMiddle + d : B::kMiddle - d], 1u);
    return B::kSingle && unsigned(d - 1) >= unsigned(B::kFine);
  };
  row.template each<kThreads>(
      [&](int i) {
        const float z = value_at(logits, i);
        if (z > -INFINITY && count(bits_at(logits, i))) {
          const uint32_t k = atomicAdd(&sh->mine, 1u);
          if (k < kAside) aside[k] = uint16_t(bits_at(logits, i));
        }
      },
      [&](const uint4& x, int) {
        uint32_t few = 0;
#pragma unroll
        for (int k = 0; k < Slice<T>::kPer; ++k) {
          if (sizeof(T) == 4 && !(value_of<T>(x, k) > -INFINITY)) continue;        // a NaN may show in the lower half alone
          few |= (count(bits_of<T>(x, k)) ? 1u : 0u) << k;
        }
        if (few) {
          uint32_t k = atomicAdd(&sh->mine, uint32_t(__popc(few)));
#pragma unroll
          for (int e = 0; e < Slice<T>::kPer; ++e)
            if ((few >> e) & 1u) {
              if (k < kAside) aside[k] = uint16_t(bits_of<T>(x, e));
              ++k;
            }
        }
      });
  __syncthreads();

  // ---- places by count
  const int bin0 = min(tid * kPer, B::kCount), bin1 = min(bin0 + kPer, B::kCount);
  uint32_t count0 = 0, total;
  uint64_t weight0 = 0, all;
  for (int i = bin0; i < bin1; ++i) count0 += bin_count[i];
  const uint32_t mine = count0;
  scan<kThreads>(sh, count0, weight0, total, all);
  uint32_t enough = total;                 // n_m
  if (S.by_m) {
    const float least = S.least;
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
    scan<kThreads>(sh, n, none, enough, all);
    if (__syncthreads_or(cut)) {
      // the bin that the limit falls into, element by element
      each_logit<kThreads>(row, [&](uint32_t bits, float z, int) {
        if (z >= least && B::low_key(B::of(bits)) < key) ++zero;
      });
      uint32_t more;
      none = 0;
      scan<kThreads>(sh, zero, none, more, all);
      enough += more;
    }
    enough = max(enough, 1u);
  }
  const uint32_t most = S.top_k > 0 ? min(uint32_t(S.top_k), total) : total;
  const bool by_p = S.by_p;
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
  if (__syncthreads_or(several)) {
    if constexpr (B::kSingle) {
      // three sums: in registers, then a warp at a time
      uint64_t w[3] = {0ull, 0ull, 0ull};
      auto add = [&](uint32_t bits, float z, int) {
        const int i = B::of(bits);
        if (i <= last_bin && !B::single(i)) {
          const uint64_t x = weigh(z);
          if (i == 0) w[0] += x;
          else if (i == B::kMiddle) w[1] += x;
          else w[2] += x;
        }
      };
      if (sh->mine <= kAside)
        for (int k = tid; k < int(sh->mine); k += kThreads) add(aside[k], to_float<T>(aside[k]), 0);
      else
        each_logit<kThreads>(row, add);
      for (int k = 0; k < 3; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w[k] += __shfl_xor_sync(kFull, w[k], o);
        if (lane == 0 && w[k]) atomicAdd(reinterpret_cast<unsigned long long*>(&bin_weight[k]), (unsigned long long)w[k]);
      }
    } else {
      each_logit<kThreads>(row, [&](uint32_t bits, float z, int) {
        const int i = B::of(bits);
        if (i <= last_bin) atomicAdd(reinterpret_cast<unsigned long long*>(&bin_weight[i]), (unsigned long long)weigh(z));
      });
    }
  }
  __syncthreads();
  auto weight_of = [&](int i) -> uint64_t {
    const uint32_t n = bin_count[i];
    if (n == 0) return 0ull;
    return B::single(i) ? n * weigh(B::value(i)) : bin_weight[slot(i)];
  };
  weight0 = 0;
  if constexpr (B::kSingle) {
    // Neighbours of one exponent lie one step apart, so each weight is the last one times the
    // same factor: a product instead of a power.  Taken afresh at least every 16 bins, so that
    // the factor's error, 2^-46.5, does not add up to more than 2^-42.5 (2^-43.8 is the most seen).
    int exponent = -1, steps = 0;
    uint64_t w = 0, factor = 0;
    const int end = mine > 0 ? min(bin1, last_bin + 1) : bin0;
    for (int i = bin0; i < end; ++i) {
      const uint32_t n = bin_count[i];
      if (!B::single(i)) {
        if (n > 0) weight0 += bin_weight[slot(i)];
        exponent = -1;
        continue;
      }
      const uint32_t bits = B::bits(i);
      const int e = B::exponent(bits);
      if (e != exponent || ++steps == 16) {
        if (B::value(i) > weigh.top) continue;     // nothing lies there, and no weight to go on from
        w = weigh.fine(B::value(i));
        if (e != exponent) factor = weigh.ratio(B::step(bits));
        exponent = e;
        steps = 0;
      } else {
        w = __umul64hi(w, factor);
      }
      weight0 += n * weigh.rounded(w);
    }
  } else {
    for (int i = bin0; i < min(bin1, last_bin + 1); ++i) weight0 += weight_of(i);
  }
  uint64_t own = weight0;
  {
    uint32_t c = 0, cc;
    scan<kThreads>(sh, c, weight0, cc, all);
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
    // every warp looks at that thread's bins.  (The sum over a thread's bins may be some last
    // bits more than that of its bins one by one: then the last of them takes what is left.)
    const int end = min(bin + kPer, B::kCount);
    int last = bin;
    Place last_at = at;
    uint64_t last_weight = 0;
    bool found = false;
    for (int i0 = bin; i0 < end && !found; i0 += 32) {
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
      const uint32_t some = __ballot_sync(kFull, by_count ? c1 > 0 : w1 > 0);
      found = hit != 0;
      if (hit || some) {
        const int l = hit ? __ffs(hit) - 1 : 31 - __clz(some);
        last = i0 + l;
        last_at.count = at.count + __shfl_sync(kFull, c - c1, l);
        last_at.weight = at.weight + __shfl_sync(kFull, w - w1, l);
        last_weight = __shfl_sync(kFull, w1, l);
      }
      at.count += __shfl_sync(kFull, c, 31);
      at.weight += __shfl_sync(kFull, w, 31);
    }
    bin = last;
    at = last_at;
    if (!found) x = at.weight + last_weight - 1;
    at.key = B::high_key(bin);
    if (!B::single(bin)) {
      // divided again until a part is one value
      uint32_t lo = B::low_key(bin), hi = at.key;
      for (;;) {
        const uint32_t span = hi - lo;
        const int bits = span ? 32 - __clz(span) : 0, down = bits > 11 ? bits - 11 : 0;
        __syncthreads();
        for (int i = tid; i < kParts; i += kThreads) {
          parts->count[i] = 0;
          parts->weight[i] = 0;
        }
        __syncthreads();
        each_logit<kThreads>(row, [&](uint32_t, float z, int) {
          const uint32_t key = ord_f32(z);
          if (key >= lo && key <= hi) {
            const uint32_t i = (hi - key) >> down;
            atomicAdd(&parts->count[i], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&parts->weight[i]), (unsigned long long)weigh(z));
          }
        });
        __syncthreads();
        constexpr int kEach = kParts / kThreads;
        uint32_t c = 0, cc;
        uint64_t w = 0, ww;
        for (int k = 0; k < kEach; ++k) {
          c += parts->count[tid * kEach + k];
          w += parts->weight[tid * kEach + k];
        }
        scan<kThreads>(sh, c, w, cc, ww);
        c += at.count;
        w += at.weight;
        for (int k = 0; k < kEach; ++k) {
          const uint32_t n = parts->count[tid * kEach + k];
          const uint64_t m = parts->weight[tid * kEach + k];
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
    const uint64_t reach = share_of(sum, S.top_p, true);             // at least 1: p > 0
    const Place end = find(false, reach - 1);
    n = end.count + end.r + 1;
    sum = upto(end);
  }
  if (enough < n) {
    n = enough;
    sum = upto(find(true, n - 1));
  }
  const uint64_t x = min(share_of(sum, S.u, false), sum - 1);
  const Place drawn = find(false, x);

  // ---- the drawn.r-th token (from 0) of that logit in the order of ids
  const float z = unord_f32(drawn.key);
  constexpr int kVec = Slice<T>::kPer;
  const int head = row.head, tail = row.tail, vecs = row.v1;
  const uint4* body = row.body;
  auto matches = [&](const uint4& x) -> uint32_t {           // a bit for each element of a vector
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kVec; ++k) m |= (value_of<T>(x, k) == z ? 1u : 0u) << k;
    return m;
  };
  // warp w has the vectors from w share to (w + 1) share; the head is before them, the tail behind
  const int share = (vecs + (kThreads / 32) - 1) / (kThreads / 32), v0 = min(warp * share, vecs), v1 = min(v0 + share, vecs);
  uint32_t hits = 0;
  for (int v = v0 + lane; v < v1; v += 32 * 4) {
    uint4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + 32 * k < v1) x[k] = __ldg(body + v + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (v + 32 * k < v1) hits += __popc(matches(x[k]));
  }
  hits = __reduce_add_sync(kFull, hits);
  __syncthreads();
  if (lane == 0) sh->warp_count[warp] = hits;
  __syncthreads();
  if (warp != 0) return;
  uint32_t left = drawn.r;
  int token = -1;
  auto singly = [&](int i0, int i1) {
    for (int i = i0; i < i1 && token < 0; ++i)
      if (float(logits[i]) == z) {
        if (left == 0) token = i;
        else --left;
      }
  };
  singly(0, head);
  if (token < 0) {
    int w = 0;
    while (w < (kThreads / 32) && left >= sh->warp_count[w]) left -= sh->warp_count[w++];
    if (w < (kThreads / 32)) {
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
    P.tokens[at] = token;
    P.probs[at] = ratio(weigh(unord_f32(drawn.key)), sum);
  }
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of a variable of this CTA in another one of the cluster.
__device__ __forceinline__ uint32_t there(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void put32(uint32_t at, uint32_t x) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ void put64(uint32_t at, uint64_t x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(at), "l"(x) : "memory");
}
__device__ __forceinline__ uint32_t get32(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t add32(uint32_t at, uint32_t x) {
  uint32_t old;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(x) : "memory");
  return old;
}

// ------------------------------------------------------------------- the list
// Descending, by all threads; n <= kList, entries behind it are cleared up to a power of two.
template <int NT>
__device__ __forceinline__ void sort_list(uint64_t* list, int n) {
  const int tid = threadIdx.x;
  int N = 32;
  while (N < n) N <<= 1;
  for (int i = n + tid; i < N; i += NT) list[i] = 0;
  __syncthreads();
  if (N <= NT) {                       // an entry a thread; within a warp by shuffles
    uint64_t x = tid < N ? list[tid] : 0ull;
    for (int size = 2; size <= N; size <<= 1) {
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        uint64_t y;
        if (stride < 32) {
          if (tid >= N) continue;
          y = __shfl_xor_sync(kFull, x, stride);
        } else {
          __syncthreads();
          if (tid < N) list[tid] = x;
          __syncthreads();
          if (tid >= N) continue;
          y = list[tid ^ stride];
        }
        const bool keep_max = ((tid & stride) == 0) == ((tid & size) == 0);
        if ((x < y) == keep_max) x = y;
      }
    }
    __syncthreads();
    if (tid < N) list[tid] = x;
  } else {
    for (int size = 2; size <= N; size <<= 1) {
      for (int stride = size >> 1; stride > 0; stride >>= 1) {
        for (int i = tid; i < N / 2; i += NT) {
          const int a = 2 * i - (i & (stride - 1)), b = a + stride;
          const uint64_t x = list[a], y = list[b];
          if ((x < y) == ((a & size) == 0)) {
            list[a] = y;
            list[b] = x;
          }
        }
        __syncthreads();
      }
    }
  }
  __syncthreads();
}

// Sum over the CTA's threads, to all of them.
template <int NT>
__device__ __forceinline__ uint32_t block_sum(Shared* sh, uint32_t x) {
  x = __reduce_add_sync(kFull, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh->warp_count[threadIdx.x >> 5] = x;
  __syncthreads();
  return __reduce_add_sync(kFull, (threadIdx.x & 31) < NT / 32 ? sh->warp_count[threadIdx.x & 31] : 0u);
}

// What the list of n tokens decides: the row's draw (kDone), how far the list has to reach
// (kPlan, with sh->want), or nothing (kGeneral).
// above, below: the weights of the tokens before the list and behind it, together off by at
// most `slack`; complete: there are none.  known: the sum of what is kept, once it is known
// (then x is drawn from it); it receives that sum.
template <int NT>
__device__ __forceinline__ Verdict decide(const Settings& S, const Weigh& weigh, Shared* sh, const uint64_t* list,
                                          uint64_t* cum, int n, uint64_t above, uint64_t below, uint64_t slack,
                                          bool complete, float cut, uint64_t& known, int32_t* token, float* prob) {
  constexpr int kEach = kList / NT;
  const int tid = threadIdx.x, each = (n + NT - 1) / NT, i0 = tid * each;
  uint64_t run[kEach], w = 0, head;
  uint32_t c = 0, cc, kept = 0;
  for (int e = 0; e < kEach; ++e) {
    run[e] = 0;
    if (e < each && i0 + e < n) {
      const float z = unord_f32(uint32_t(list[i0 + e] >> 32));
      w += weigh(z);
      kept += z >= S.least;
    }
    run[e] = w;
  }
  scan<NT>(sh, c, w, cc, head);
  head += above;
  for (int e = 0; e < kEach; ++e) {
    run[e] += w + above;
    if (e < each && i0 + e < n) cum[i0 + e] = run[e];
  }
  // tokens of the list whose running sum is at most x
  auto upto = [&](uint64_t x) {
    if (each <= 1) return int(__syncthreads_count(tid < n && run[0] <= x));
    uint32_t k = 0;
    for (int e = 0; e < kEach; ++e) k += e < each && i0 + e < n && run[e] <= x;
    return int(block_sum<NT>(sh, k));
  };
  // Whether the first running sum above x lies in the list whatever the sums that are off;
  // if not, how far it is.
  const float units = __uint_as_float(uint32_t(127 - weigh.shift) << 23);
  auto place = [&](uint64_t x, int& i) {
    i = upto(x);
    bool sure = i < n && (above == 0 || x >= above);
    if (slack > 0)
      sure = sure && x + slack < head && (above == 0 || x >= above + slack) && upto(x > slack ? x - slack : 0ull) == i &&
             upto(x + slack) == i;
    if (!sure && tid == 0) {
      sh->want = float(x) * units;
      sh->behind = float(head + below - x) * units;
    }
    return sure;
  };
  int keep = n, i;
  uint64_t sum = known ? known : head + below;
  if (known == 0) {
    if (S.by_k) {
      if (n < S.top_k && !complete && !(S.by_m && !S.by_p)) {
        if (tid == 0) sh->want = float(S.top_k);
        return kPlan;
      }
      keep = min(n, S.top_k);
      __syncthreads();
      sum = cum[keep - 1];
    }
    // tokens that min-p keeps; all of them are listed where the list goes down to its limit
    const int most = S.by_m ? max(1, each <= 1 ? int(__syncthreads_count(kept)) : int(block_sum<NT>(sh, kept))) : n;
    if (S.by_p) {
      const uint64_t x = share_of(sum, S.top_p, true) - 1;             // at least 1: p > 0
      if (place(x, i)) keep = min(keep, i + 1);
      // wherever the share is reached, min-p ends before it
      else if (!(S.by_m && S.least >= cut && above == 0 && x >= slack && upto(x - slack) >= most)) return kPlan;
    }
    if (S.by_m) keep = min(keep, most);
    if (S.by_p || S.by_m) {
      __syncthreads();
      sum = cum[keep - 1];
      if (above == 0) slack = 0;
    }
  }
  if (!place(min(share_of(sum, S.u, false), sum - 1), i)) {
    if (S.by_p && known == 0) known = sum;
    return kPlan;
  }
  if (tid == 0) {
    i = min(i, keep - 1);
    *token = int32_t(~uint32_t(list[i]));
    *prob = ratio(cum[i] - (i > 0 ? cum[i - 1] : above), sum);
  }
  return kDone;
}

// decide() for a list of at most 128 tokens before which nothing lies, by one warp, in its
// registers: token 32 e + lane is the lane's e-th.  Nothing waits for another warp.
constexpr int kShort = 128;
__device__ __forceinline__ Verdict decide_short(const Settings& S, const Weigh& weigh, Shared* sh, const uint64_t* list,
                                                int n, uint64_t below, uint64_t slack, bool complete, float cut,
                                                int32_t* token, float* prob) {
  constexpr int E = kShort / 32;
  const int lane = threadIdx.x & 31, used = (n + 31) / 32;
  int N = 32;
  while (N < n) N <<= 1;
  uint64_t x[E], run[E];
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = 32 * e + lane < n ? list[32 * e + lane] : 0ull;
  for (int size = 2; size <= N; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      if (stride < 32) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (32 * e >= N) break;
          const uint64_t y = __shfl_xor_sync(kFull, x[e], stride);
          const bool keep_max = ((lane & stride) == 0) == (((32 * e + lane) & size) == 0);
          if ((x[e] < y) == keep_max) x[e] = y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int o = e ^ (stride >> 5);
          if (o > e && 32 * o < N) {
            // entries of this and the other register in one lane
#pragma unroll
            for (int f = 0; f < E; ++f)
              if (f == o) {
                const bool down = ((32 * e) & size) == 0;
                const uint64_t a = x[e], b = x[f];
                if ((a < b) == down) {
                  x[e] = b;
                  x[f] = a;
                }
              }
          }
        }
      }
    }
  }
  uint64_t head = 0;
  int kept = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    run[e] = 0;
    if (e >= used) continue;
    const bool on = 32 * e + lane < n;
    const float z = unord_f32(uint32_t(x[e] >> 32));
    uint64_t w = on ? weigh(z) : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w += y;
    }
    run[e] = head + w;
    head += __shfl_sync(kFull, w, 31);
    kept += __popc(__ballot_sync(kFull, on && z >= S.least));
  }
  auto upto = [&](uint64_t v) {
    int k = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < used) k += __popc(__ballot_sync(kFull, 32 * e + lane < n && run[e] <= v));
    return k;
  };
  auto sum_at = [&](int i) {                 // the running sum with token i
    uint64_t v = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e == (i >> 5)) v = __shfl_sync(kFull, run[e], i & 31);
    return v;
  };
  const float units = __uint_as_float(uint32_t(127 - weigh.shift) << 23);
  auto place = [&](uint64_t v, int& i) {
    i = upto(v);
    bool sure = i < n;
    if (slack > 0) sure = sure && v + slack < head && upto(v > slack ? v - slack : 0ull) == i && upto(v + slack) == i;
    if (!sure && lane == 0) {
      sh->want = float(v) * units;
      sh->behind = float(head + below - v) * units;
    }
    return sure;
  };
  int keep = n, i;
  uint64_t sum = head + below;
  if (S.by_k) {
    if (n < S.top_k && !complete && !(S.by_m && !S.by_p)) {
      if (lane == 0) sh->want = float(S.top_k);
      return kPlan;
    }
    keep = min(n, S.top_k);
    sum = sum_at(keep - 1);
  }
  const int most = S.by_m ? max(1, kept) : n;
  if (S.by_p) {                              // as in decide()
    const uint64_t v = share_of(sum, S.top_p, true) - 1;
    if (place(v, i)) keep = min(keep, i + 1);
    else if (!(S.by_m && S.least >= cut && v >= slack && upto(v - slack) >= most)) return kPlan;
  }
  if (S.by_m) keep = min(keep, most);
  if (S.by_p || S.by_m) {
    sum = sum_at(keep - 1);
    slack = 0;
  }
  if (!place(min(share_of(sum, S.u, false), sum - 1), i)) return kPlan;
  i = min(i, keep - 1);
  const uint64_t to = sum_at(i), w = to - (i > 0 ? sum_at(i - 1) : 0ull);
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (32 * e + lane == i) {
      *token = int32_t(~uint32_t(x[e]));
      *prob = ratio(w, sum);
    }
  return kDone;
}

// Largest of a vector's elements, NaN left out (two of them where they have 16 bits).
template <typename T> __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b);
template <> __device__ __forceinline__ uint32_t max2<__nv_bfloat16>(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
template <> __device__ __forceinline__ uint32_t max2<__half>(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
template <typename T> constexpr uint32_t kLowest2 = 0xFF7FFF7Fu;        // the lowest finite value, twice
template <> constexpr uint32_t kLowest2<__half> = 0xFBFFFBFFu;
template <typename T> constexpr uint32_t kNone2 = 0xFF80FF80u;          // -inf, twice
template <> constexpr uint32_t kNone2<__half> = 0xFC00FC00u;
template <typename T>
__device__ __forceinline__ float max_of(const uint4& x) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t m = max2<T>(max2<T>(x.x, x.y), max2<T>(x.z, x.w));
    return fmaxf(to_float<T>(m & 0xFFFFu), to_float<T>(m >> 16));
  } else {
    return fmaxf(fmaxf(__uint_as_float(x.x), __uint_as_float(x.y)), fmaxf(__uint_as_float(x.z), __uint_as_float(x.w)));
  }
}

// Weights of tokens that are not listed, 2^-12 at most, in fp32 (u = 2^-24, half a step).  The
// exponent y is a rounded difference (u) times a factor (u by its rounding, 0.23 u by the part of
// log2(e) that is left out) in a rounded product (u), so off by 3.23 u y, and the weight by
// ln 2 of that, 2.24 u y of itself; ex2 is off by 4 u, a sum of eight by 4 u.  Together
// (2.24 y + 8) u: 2^-17 of the weight up to y = 53.  A weight beyond that is less than a part, as
// rows with a list have more than 256 tokens and parts of 2^-53 or more, and its error, 2^-16.7 of
// it up to y = 64, next to nothing.  A vector's sum is rounded to a whole part, half of one for
// four tokens or more (the few outside vectors one by one), and what stands in for a listed token
// weighs less than 2^-10 of a part.  So a row's sum is within 2^-17 of itself and V parts: the guard
// band of a list that is not complete.
template <typename T>
struct Tail {
  float top, c, one;                         // one: 2^shift
  __device__ __forceinline__ uint64_t operator()(const uint4& x) const {
    const uint64_t low2 = pair(-top, -top), c2 = pair(c, c);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint64_t sum = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t v = max2<T>(w[k], kLowest2<T>);                 // -inf and NaN weigh nothing
        const uint64_t y = mul2(add2(pair(to_float<T>(v & 0xFFFFu), to_float<T>(v >> 16)), low2), c2);
        sum = add2(sum, pair(ex2_approx(low(y)), ex2_approx(high(y))));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float a = fmaxf(__uint_as_float(w[k]), -3.4028235e38f), b = fmaxf(__uint_as_float(w[k + 1]), -3.4028235e38f);
        const uint64_t y = mul2(add2(pair(a, b), low2), c2);
        sum = add2(sum, pair(ex2_approx(low(y)), ex2_approx(high(y))));
      }
    }
    return __float2ull_rn((low(sum) + high(sum)) * one);
  }
  __device__ __forceinline__ uint64_t operator()(float z) const { return __float2ull_rn(ex2_approx((z - top) * c) * one); }
};

constexpr int kSteps = 64;                   // of a plan, in a binary order of weight
constexpr float kNear = 12.f;                // binary orders that are listed at first
constexpr int32_t kUndecided = -2, kTaken = -3;    // a row's token until general() has drawn it

// The settings of a row's sequence, and the weights' factor: log2(e) / heat in two parts,
// each step's remainder carried on.
struct Asked {
  Settings S;
  bool greedy;
  float c_hi, c_lo;
};
__device__ __forceinline__ Asked settings_of(const SampleParams& P, long long at, int V) {
  const int b = int(at / P.R);
  Asked a;
  Settings& S = a.S;
  S.heat = P.temperature ? P.temperature[b] : 1.f;
  S.top_k = P.top_k ? P.top_k[b] : 0;
  S.top_p = P.top_p ? P.top_p[b] : 1.f;
  S.min_p = P.min_p ? P.min_p[b] : 0.f;
  S.u = P.uniforms[at];
  S.by_k = S.top_k > 0 && S.top_k < V;
  S.by_p = S.top_p < 1.f;
  S.by_m = S.min_p > 0.f;
  S.tail = !S.by_k && (S.by_p || !S.by_m);
  S.least = -INFINITY;
  a.greedy = !(S.heat > 0.f) || S.top_k == 1 || S.top_p <= 0.f || S.min_p > 1.f;
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-8f;   // log2(e)
  a.c_hi = kHi / S.heat;
  a.c_lo = (fmaf(-a.c_hi, S.heat, kHi) + kLo) / S.heat;
  if (!(a.c_hi < 1e30f)) {                   // every logit but the largest weighs nothing anyway
    a.c_hi = 1e30f;
    a.c_lo = 0.f;
  }
  if (!(S.heat < INFINITY)) a.c_hi = a.c_lo = 0.f;
  return a;
}
__device__ __forceinline__ void fill_table(Shared* sh) {
  if (threadIdx.x < 256)
    sh->table[threadIdx.x] = __umul64hi(kSixteenths[threadIdx.x >> 4], kParts256[threadIdx.x & 15]) >> 1;
}
// w >= min_p where z >= max + T ln(min_p); by one thread, in 64 bits.
__device__ __forceinline__ float least_of(const Settings& S, float top) {
  const float x = __double2float_ru(double(top) + double(S.heat) * log(double(S.min_p)));
  return x <= top ? x : -INFINITY;           // an infinite temperature times nothing
}

// NT threads; kAll: a row that the list does not decide goes by general() here, else its token
// becomes kUndecided and rest_kernel draws it.
template <typename T, int NT, int kCtas, bool kAll>
__global__ void __launch_bounds__(NT, kCtas) sample_kernel(const SampleParams P) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared* sh = reinterpret_cast<Shared*>(smem);
  uint64_t* list = reinterpret_cast<uint64_t*>(sh + 1);
  uint64_t* cum = list + kList;
  uint32_t* plan = reinterpret_cast<uint32_t*>(cum);                   // kList counts
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ranks = kAll ? uint32_t(P.ranks) : 1u, rank = kAll && ranks > 1 ? cluster_rank() : 0u;
  const long long at = blockIdx.x / ranks;                             // the row
  const int V = P.V;
  const T* logits = static_cast<const T*>(P.logits) + at * P.stride;
  const Slice<T> row(logits, V, int(rank), int(ranks));
  auto sync = [&]() {
    if (kAll && ranks > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  if (tid == 0) {
    sh->mine = 0;
    sh->others = 0;
    sh->first = 0xFFFFFFFFu;
  }
  if (kAll && ranks > 1) cluster_arrive();   // every CTA runs before another one writes to it
  const Asked asked = settings_of(P, at, V);
  Settings S = asked.S;
  const bool greedy = asked.greedy;
  const float lowest = -3.4028235e38f;
  // a binary order of weight in logits
  const float binary = fminf(0.69314718055994531f * S.heat, 3.4028235e38f);

  // ---- the largest logit, and those of the thread's eight parts of the row
  constexpr int kGroups = 8;
  float most[kGroups], mine = -INFINITY;
  uint32_t most2[kGroups];                   // two at a time where they have 16 bits
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    most[u] = -INFINITY;
    most2[u] = kNone2<T>;
  }
  for (int v = row.v0 + tid; v < row.v1; v += NT * kGroups) {
    uint4 x[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
      if (v + u * NT < row.v1) x[u] = __ldg(row.body + v + u * NT);
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
      if (v + u * NT < row.v1) {
        if constexpr (sizeof(T) == 2) most2[u] = max2<T>(most2[u], max2<T>(max2<T>(x[u].x, x[u].y), max2<T>(x[u].z, x[u].w)));
        else most[u] = fmaxf(most[u], max_of<T>(x[u]));
      }
  }
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int u = 0; u < kGroups; ++u) most[u] = fmaxf(to_float<T>(most2[u] & 0xFFFFu), to_float<T>(most2[u] >> 16));
  }
  if (row.first && tid < row.head) most[0] = fmaxf(most[0], value_at(logits, tid));
  if (row.last && row.tail + tid < V) most[0] = fmaxf(most[0], value_at(logits, row.tail + tid));
#pragma unroll
  for (int u = 0; u < kGroups; ++u) mine = fmaxf(mine, most[u]);
  float top;
  uint32_t best = __reduce_max_sync(kFull, ord_f32(mine));
  if (lane == 0) sh->warp_count[warp] = best;
  if (!greedy) fill_table(sh);
  __syncthreads();
  best = __reduce_max_sync(kFull, sh->warp_count[lane % (NT / 32)]);
  // What top_k of the maxima of disjoint parts of the row reach is reached by top_k tokens:
  // the list need not go further down.  CTAs that share a row each look for their part of
  // top_k, and the lowest answer holds for all.
  uint32_t reach = 0;
  const int enough_here = (S.top_k + int(ranks) - 1) / int(ranks);
  if (!greedy && S.by_k && enough_here <= kGroups / 2 * NT) {
    float lo = fmaxf(unord_f32(best) - 32.f * binary, lowest), hi = unord_f32(best);
    auto enough = [&](float x) {
      uint32_t n = 0;
#pragma unroll
      for (int u = 0; u < kGroups; ++u) n += most[u] >= x;
      return int(block_sum<NT>(sh, n)) >= enough_here;
    };
    if (enough(lo)) {
      for (int i = 0; i < 10; ++i) {
        const float mid = 0.5f * (lo + hi);
        if (enough(mid)) lo = mid;
        else hi = mid;
      }
      reach = ord_f32(lo);
    }
  }
  if (kAll && ranks > 1) {
    cluster_wait();
    if (tid < int(ranks)) put64(there(&sh->tops[rank], tid), uint64_t(best) << 32 | reach);
    sync();
    const uint64_t x = sh->tops[lane % ranks];
    best = __reduce_max_sync(kFull, uint32_t(x >> 32));
    reach = __reduce_min_sync(kFull, uint32_t(x));       // 0 where one of them has none
  }
  top = unord_f32(best);
  if (top == -INFINITY) {                    // nothing is left to draw from
    if (rank == 0 && tid == 0) {
      P.tokens[at] = -1;
      P.probs[at] = 0.f;
    }
    return;
  }

  // The row again, from its end on (the rows of all CTAs may be more than the L2 holds, and what was
  // read last is still there); where what lies below z does not count, only those of the thread's
  // eight parts of it that have a logit from z on (4 x 497 rows of 151936: top-k 210 us for 180).
  auto again = [&](bool whole, float z, auto&& one, auto&& vec) {
    constexpr int kUnroll = 4;
    if (row.first && tid < row.head) one(tid);
    if (row.last && row.tail + tid < V) one(row.tail + tid);
    uint32_t parts = whole ? 1u : 0u;
#pragma unroll
    for (int u = 0; u < kGroups; ++u) parts |= (!whole && most[u] >= z ? 1u : 0u) << u;
    const int stride = whole ? NT : NT * kGroups, step = kUnroll * stride;
    while (parts) {
      const int from = row.v0 + (__ffs(parts) - 1) * NT + tid;
      parts &= parts - 1;
      for (int v = from + (max(row.v1 - from - 1, 0) / step) * step; v >= from; v -= step) {
        uint4 x[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (v + i * stride < row.v1) x[i] = __ldg(row.body + v + i * stride);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
          if (v + i * stride < row.v1) vec(x[i], row.head + (v + i * stride) * Slice<T>::kPer);
      }
    }
  };

  if (greedy) {
    uint32_t first = 0xFFFFFFFFu;
    again(false, top, [&](int i) { if (value_at(logits, i) == top) first = min(first, uint32_t(i)); },
              [&](const uint4& x, int i) {
                if (max_of<T>(x) != top) return;
#pragma unroll
                for (int k = Slice<T>::kPer - 1; k >= 0; --k)
                  if (value_of<T>(x, k) == top) first = min(first, uint32_t(i + k));
              });
    if (first != 0xFFFFFFFFu) atomicMin(&sh->first, first);
    __syncthreads();
    first = sh->first;
    if (kAll && ranks > 1) {
      if (tid == 0) put64(there(&sh->tails[rank], 0), first);
      sync();
      if (rank != 0) return;
      first = __reduce_min_sync(kFull, uint32_t(sh->tails[lane % ranks]));
    }
    if (tid == 0) {
      P.tokens[at] = int32_t(first);
      P.probs[at] = 1.f;
    }
    return;
  }

  Weigh weigh;
  weigh.top = top;
  weigh.shift = P.shift;
  weigh.table = sh->table;
  weigh.c_hi = asked.c_hi;
  weigh.c_lo = asked.c_lo;
  if (S.by_m) {
    if (tid == 0) sh->least = least_of(S, top);
    __syncthreads();
    S.least = sh->least;
  }
  S.tail = S.tail && top < INFINITY;
  const Tail<T> light{top, weigh.c_hi, __uint_as_float(uint32_t(127 + P.shift) << 23)};
  // short rows are listed whole; min-p alone says itself what is kept
  float cut = fmaxf(top - kNear * binary, lowest);
  // the type's lowest value, which stands for none below, has to weigh nothing
  if (V <= NT || top - to_float<T>(kLowest2<T> & 0xFFFFu) < 64.f * binary) cut = lowest;
  else if (top == INFINITY) cut = top;
  else if (reach != 0) cut = unord_f32(reach);
  if (V > NT && S.by_m && !S.by_p) cut = fmaxf(S.by_k && reach != 0 ? fmaxf(cut, S.least) : S.least, lowest);
  const Mid& mid = weigh;
  uint64_t known = 0;

  // ---- the tokens near the largest, and the weight of the others
  uint64_t before = 0, behind = 0;
  const bool rest_counts = S.tail && cut > lowest;
  auto put = [&](float z, int i, uint32_t k) {
    if (k < uint32_t(kList)) list[k] = elem_key(z, uint32_t(i));
  };
  auto list_one = [&](int i) {
    const float z = value_at(logits, i);
    if (z >= cut) put(z, i, atomicAdd(&sh->mine, 1u));
    else if (rest_counts && z > -INFINITY) behind += light(z);
  };
  auto list_vec = [&](const uint4& x, int i) {
    if (max_of<T>(x) < cut) {
      if (rest_counts) behind += light(x);
      return;
    }
    uint32_t hits = 0;
    uint4 y = x;                         // without the hits
#pragma unroll
    for (int k = 0; k < Slice<T>::kPer; ++k)
      if (value_of<T>(x, k) >= cut) {
        hits |= 1u << k;
        uint32_t& w = (k * int(sizeof(T)) / 4 == 0) ? y.x : (k * int(sizeof(T)) / 4 == 1) ? y.y : (k * int(sizeof(T)) / 4 == 2) ? y.z : y.w;
        w = sizeof(T) == 4 ? 0xFF7FFFFFu : k & 1 ? (w & 0xFFFFu) | (kLowest2<T> & 0xFFFF0000u) : (w & 0xFFFF0000u) | (kLowest2<T> & 0xFFFFu);
      }
    if (rest_counts) behind += light(y);
    if (hits) {
      uint32_t k = atomicAdd(&sh->mine, uint32_t(__popc(hits)));
      do {
        const int e = __ffs(hits) - 1;
        hits &= hits - 1;
        put(value_at(logits, i + e), i + e, k++);
      } while (hits);
    }
  };
  again(rest_counts, cut, list_one, list_vec);
  // Whether a list that does not decide is made again where a plan says: of 16-bit logits
  // general() is quicker (100 thousand cycles for 200 with 32000 of them).  It was not for the first
  // top_k of a large vocabulary before the maxima bounded lists up to 1024, which need no plan now.
  // What is left for this rule, top_k above that, mostly loses by it (plan for general(); 1988 rows of
  // 151936: bf16, top_k 2000 1250..1286 us for 944..986, fp16 1129..1312 for 1214..1271, top_k 8000
  // 1499..1547 for 1227..1270; of 66000, bf16 738..815 for 519..540; top_k 1000 473..476 for 468..472).
  const bool plans = sizeof(T) == 4 || (ranks == 1 && S.by_k && V > 65536);
  bool planned = false;
  for (;;) {
    // ---- the list and the sums come together, and what they decide
    uint64_t above = 0, below = 0;
    if (S.tail) {
      uint32_t z = 0, zz;
      if (planned) scan<NT>(sh, z, before, zz, above);
      scan<NT>(sh, z, behind, zz, below);
    }
    __syncthreads();
    int n = int(min(sh->mine, uint32_t(2 * kList)));
    if (kAll && ranks > 1) {
      if (rank != 0) {
        // hand it over: one place is asked for, then all entries are written
        if (tid == 0) {
          sh->at_count = add32(there(&sh->others, 0), uint32_t(n));
          put64(there(&sh->tails[rank], 0), below);
          put64(there(&sh->heads[rank], 0), above);
        }
        __syncthreads();
        const uint32_t from = sh->at_count;
        for (int i = tid; i < min(n, kList); i += NT)
          if (from + i < uint32_t(kList)) put64(there(&cum[from + i], 0), list[i]);
      }
      sync();
      // what a row of 16-bit logits needs beyond its list, the first CTA does alone
      if (rank != 0 && sizeof(T) == 2) return;
      if (rank == 0) {
        const int others = int(sh->others);
        if (n + others <= kList)
          for (int i = tid; i < others; i += NT) list[n + i] = cum[i];
        n += others;
        for (uint32_t r = 1; r < ranks; ++r) {
          below += sh->tails[r];
          above += sh->heads[r];
        }
        __syncthreads();
      }
    }
    const bool complete = cut <= lowest;
    Verdict v = kGeneral;
    if (rank == 0) {
      const bool drawing = known != 0;
      uint64_t slack = 0;
      if (S.tail && planned) slack = ((above + below + known) >> 28) + 2 * uint64_t(V);
      else if (S.tail && !complete) slack = (below >> 17) + uint64_t(V);
      if (n <= kShort && !planned) {
        if (warp == 0) {
          v = decide_short(S, weigh, sh, list, n, below, slack, complete, cut, &P.tokens[at], &P.probs[at]);
          if (lane == 0) {
            if (!kAll && !plans && v != kDone) {
              P.tokens[at] = kUndecided;
              P.probs[at] = top;
            }
            sh->verdict = v;
          }
        }
        if (!kAll && !plans) return;
        __syncthreads();
        v = Verdict(sh->verdict);
        __syncthreads();                     // read before it is written again
      } else if (n <= kList && n > 0) {
        sort_list<NT>(list, n);
        v = decide<NT>(S, weigh, sh, list, cum, n, above, below, slack, complete && above == 0, cut, known, &P.tokens[at],
                       &P.probs[at]);
      } else if (!planned && !(S.by_m && !S.by_p)) {
        v = kPlan;                           // by what the histogram says
        if (tid == 0) sh->want = S.by_k ? float(S.top_k) : -1.f;
      }
      // once more at most for the share, and once for the draw
      if (v == kPlan && planned && (drawing || known == 0)) v = kGeneral;
      if (v == kPlan && !plans) v = kGeneral;
    }
    // ---- how far down the list has to go: counts by distance from the largest
    float from = 0.f, scale = float(kSteps);
    uint64_t base = 0, after = 0;            // the weights before and behind a plan's steps, here in parts of 2^-38 of the largest
    for (int level = 0;; ++level) {
      if (kAll && ranks > 1 && sizeof(T) != 2) {
        if (rank == 0 && tid < int(ranks)) {
          put32(there(&sh->verdict, tid), v);
          put32(there(&sh->from, tid), __float_as_uint(from));
          put32(there(&sh->scale, tid), __float_as_uint(scale));
        }
        sync();
        v = Verdict(sh->verdict);
        from = sh->from;
        scale = sh->scale;
      }
      if (v != kPlan && v != kRefine) break;
      __syncthreads();
      for (int i = tid; i < kList; i += NT) plan[i] = 0;
      __syncthreads();
      each_logit<NT>(row, [&](uint32_t, float z, int) {
        const float y = ((z == top ? 0.f : (top - z) * weigh.c_hi) - from) * scale;
        if (y >= 0.f && (level == 0 || y < float(kList))) atomicAdd(&plan[y < float(kList - 1) ? int(y) : kList - 1], 1u);
      });
      sync();
      if (rank == 0) {
        constexpr int kEach = kList / NT;
        uint32_t count = 0, total, own[kEach];
        uint64_t parts = 0, all_parts;
        // a step's weight is off by half a step's 2^(1/scale) at most
        auto weight = [&](uint32_t n, int e) {
          return uint64_t(float(n) * ex2_approx(-from - (float(tid * kEach + e) + 0.5f) / scale) * 0x1p38f);
        };
        for (int e = 0; e < kEach; ++e) {
          const int i = tid * kEach + e;
          own[e] = plan[i];
          for (uint32_t r = 1; r < ranks; ++r) own[e] += get32(there(&plan[i], r));
          count += own[e];
          parts += weight(own[e], e);
        }
        scan<NT>(sh, count, parts, total, all_parts);
        // The first step that comes within 1/512 of the place, and the first that is behind it by
        // as much: of the weight before it or of the weight behind it, whichever is less (both are
        // known to more than the steps are).
        const uint64_t whole = base + all_parts + after;
        float want = sh->want, behind = sh->behind;
        if (want < 0.f) {
          want = (S.by_p ? S.top_p : fminf(fmaxf(S.u, 0.f), 1.f)) * float(whole) * 0x1p-38f;
          behind = float(whole) * 0x1p-38f - want;
        }
        const bool low = behind < want;      // then places are told by what is behind them
        const uint64_t goal = uint64_t(fmaxf(low ? behind : want, 0.f) * 0x1p38f), off = (goal >> 9) + 1;
        if (tid == 0) {
          sh->at_bin = sh->at_count = 0;
          sh->at_weight = base;
          sh->at_end = uint32_t(kList - 1);
          sh->end_count = total;
          sh->end_weight = base + all_parts;
        }
        __syncthreads();
        uint32_t c = count;
        uint64_t w = base + parts;
        for (int e = 0; e < kEach; ++e) {
          const uint64_t next = w + weight(own[e], e);
          const uint32_t upto = c + own[e];
          const bool from_here = low ? whole - w >= goal + off && whole - next < goal + off : w + off <= goal && next + off > goal;
          const bool to_here = low ? whole - w + off > goal && whole - next + off <= goal : w <= goal + off && next > goal + off;
          if (S.by_k ? c < uint32_t(S.top_k) && upto >= uint32_t(S.top_k) : to_here) {
            sh->at_end = uint32_t(tid * kEach + e);
            sh->end_count = upto;
            sh->end_weight = next;
          }
          if (!S.by_k && from_here) {
            sh->at_bin = uint32_t(tid * kEach + e);
            sh->at_count = c;
            sh->at_weight = w;
          }
          c = upto;
          w = next;
        }
        __syncthreads();
        const int end = int(sh->at_end);
        int begin = int(sh->at_bin);
        const bool beyond = end >= kList - 1;
        v = kRead;
        // from the largest on where the list can hold it, else around the place alone
        bool from_top = level == 0 && sh->end_count <= uint32_t(kList);
        float hi = NAN;                      // no logit is at least that
        if (!from_top) {
          if (S.by_k || S.by_m || begin > end) v = kGeneral;
          else if (sh->end_count - sh->at_count > uint32_t(kList)) v = level == 0 && !beyond ? kRefine : kGeneral;
          if (level > 0 || begin > 0) hi = top - (from + (float(begin) - 0.5f) / scale) * binary;
        }
        if (v == kRefine) {
          // the same steps again, 2048 parts of them
          base = sh->at_weight;
          after = whole - sh->end_weight;
          from += float(begin) / scale;
          scale *= float(kList / (end + 1 - begin));
        }
        __syncthreads();
        if (tid == 0) {
          const float to = top - (from + (float(end) + 1.5f) / scale) * binary;
          sh->cut = beyond && (level == 0) ? lowest : fmaxf(to, lowest);
          sh->cut_above = hi;
          sh->mine = 0;
          sh->others = 0;
        }
        __syncthreads();
        if (kAll && ranks > 1 && tid > 0 && tid < int(ranks)) {
          put32(there(&sh->cut, tid), __float_as_uint(sh->cut));
          put32(there(&sh->cut_above, tid), __float_as_uint(sh->cut_above));
          put32(there(&sh->mine, tid), 0u);
        }
      }
    }
    if (v == kDone) return;
    if (v == kGeneral) break;
    // ---- the list again, around that place; the sums of the others to 2^-28 and a part each
    cut = sh->cut;
    const float cut_above = sh->cut_above;
    planned = true;
    before = behind = 0;
    each_logit<NT>(row, [&](uint32_t, float z, int i) {
      if (z >= cut && !(z >= cut_above)) {
        put(z, i, atomicAdd(&sh->mine, 1u));
      } else if (S.tail) {
        const uint64_t w = mid(z);
        if (z < cut) behind += w;
        else before += w;
      }
    });
  }
  if (rank != 0) return;
  if constexpr (kAll) {
    general<T>(P, logits, at, weigh, S, sh, reinterpret_cast<unsigned char*>(list));
  } else if (tid == 0) {
    P.tokens[at] = kUndecided;
    P.probs[at] = top;
  }
}

// The rows that sample_kernel left undecided.  They come in runs (a sequence's settings are
// those of all of its rows), so a CTA takes one at a time, from the part of the rows that is
// its own at first and then from the others', and marks it as taken in its token; of a part's
// open rows each CTA tries another one.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) rest_kernel(const SampleParams P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ long long row;
  Shared* sh = reinterpret_cast<Shared*>(smem);
  constexpr int kEach = 4, kPart = kThreads * kEach;
  const int tid = threadIdx.x;
  const long long parts = (P.rows + kPart - 1) / kPart;
  for (long long i = 0; i < parts; ++i) {
    const long long at0 = (blockIdx.x + i) % parts * kPart;
    for (uint32_t turn = blockIdx.x;; ++turn) {
      uint32_t open = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const long long at = at0 + tid * kEach + e;
        if (at < P.rows && __ldcg(P.tokens + at) == kUndecided) open |= 1u << e;
      }
      const uint32_t here = __popc(open);
      uint32_t rank = here, total;
      uint64_t none = 0, zero;
      scan<kThreads>(sh, rank, none, total, zero);
      if (total == 0) break;
      uint32_t want = turn * 2654435761u % total;
      if (rank <= want && want < rank + here) {
        for (want -= rank; want > 0; --want) open &= open - 1;
        const long long at = at0 + tid * kEach + __ffs(open) - 1;
        row = atomicCAS(P.tokens + at, kUndecided, kTaken) == kUndecided ? at : -1;
      }
      __syncthreads();
      const long long at = row;
      if (at >= 0) {
        const Asked asked = settings_of(P, at, P.V);
        Settings S = asked.S;
        Weigh weigh;
        weigh.top = P.probs[at];
        weigh.shift = P.shift;
        weigh.table = sh->table;
        weigh.c_hi = asked.c_hi;
        weigh.c_lo = asked.c_lo;
        fill_table(sh);
        if (S.by_m && tid == 0) sh->least = least_of(S, weigh.top);
        __syncthreads();
        if (S.by_m) S.least = sh->least;
        general<T>(P, static_cast<const T*>(P.logits) + at * P.stride, at, weigh, S, sh,
                   reinterpret_cast<unsigned char*>(sh + 1));
      }
      __syncthreads();
    }
  }
}

template <typename T>
cudaError_t launch(SampleParams& P, cudaStream_t s) {
  using B = Bins<T>;
  const int bins = int(sizeof(Parts)) + 8 * (B::kSingle ? 4 : B::kCount + 1) + 4 * B::kCount, lists = 16 * kList;
  const int small = int(sizeof(Shared)) + lists, large = int(sizeof(Shared)) + (bins > lists ? bins : lists);
  const int sms = device_sms() > 0 ? device_sms() : 152;
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (P.rows <= (sizeof(T) == 4 ? 4 : 2) * sms) {
    // Large CTAs that do all for their rows, against the kernels below (us, in that order).  16 bits: 304
    // rows of 32000 83 for 106, 64 x 79 fp16 ones 368 for 311, 1988 of 151936 with all limits 189..365 for
    // 127..349.  32 bits: 500 rows of 32000 114 for 139, 608 with top-p 292 for 391, 5000 of 2000 668 for
    // 550.  The number of rows alone decides, and is not right for all: flat 16-bit rows of 32000 with
    // top-p alone would go better by the large CTAs far beyond two an SM (320 rows 90 for 111, 608 140 for
    // 175, 1988 379 for 421), 32-bit rows without top-k beyond four (2000 of 32000 476 for 589, 700 of
    // 151936 629 for 1153, with top-p 1202 for 1680; peaked ones of 32000 347 for 325), those with top-k by
    // the small ones from one an SM on (320 of 32000 31 for 23, 608 39 for 27).
    // Rows that do not fill the device are shared: as many CTAs a row as keep it to one round
    // of two an SM, none with less than 4096 logits (one row of 151936 60 us for 72 by one CTA, where
    // it goes by general(); 20 rows 110 for 109; 76 rows 115 for 107, where one CTA a row is quicker).
    const auto kernel = sample_kernel<T, kThreads, 2, true>;
    const cudaError_t e = settled(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, large));
    if (e != cudaSuccess) return e;
    P.ranks = 1;
    while (P.ranks < kMaxRanks && P.rows * 2 * P.ranks <= 2ll * sms && P.V / (2 * P.ranks) >= 4096) P.ranks *= 2;
    if (P.ranks == 1) return launch_kernel(kernel, unsigned(P.rows), kThreads, large, s, P);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(P.ranks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(unsigned(P.rows * P.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = large;
    return settled(cudaLaunchKernelEx(&cfg, kernel, static_cast<const SampleParams&>(P)));
  }
  // More rows: smaller CTAs, more of them an SM, so that one's sums and barriers pass while
  // others read; the few rows that their lists do not decide are left to a second kernel.
  const auto kernel = sample_kernel<T, kManyThreads, kManyCtas, false>;
  cudaError_t e = settled(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, small));
  if (e != cudaSuccess) return e;
  P.ranks = 1;
  e = launch_kernel(kernel, unsigned(P.rows), kManyThreads, small, s, P);
  if (e != cudaSuccess) return e;
  e = settled(cudaFuncSetAttribute(rest_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, large));
  if (e != cudaSuccess) return e;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(2 * sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = large;
  return settled(cudaLaunchKernelEx(&cfg, rest_kernel<T>, static_cast<const SampleParams&>(P)));
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
  P.R = R; P.V = V; P.rows = rows;
  P.shift = 62 - bits;                       // the sum of V weights of 1 stays below 2^62
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DART_F32   ? launch<float>(P, s)
                        : dtype == DART_F16 ? launch<__half>(P, s)
                                            : launch<__nv_bfloat16>(P, s);
  return e == cudaSuccess ? DART_OK : DART_ERR_CUDA;
}
