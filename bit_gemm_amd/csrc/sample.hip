// A token for each row of logits from given random numbers
// (include/mosaicq_head.h, mq_sample).
//
// Weights are whole numbers of 2^-40 of the largest, so sums of them are exact
// and no order of additions, split or atomic can change a result. What is kept
// is a prefix of the tokens in their order (the logit, then the index); its
// end is found by a count (top-k) and a mass (top-p): a histogram over kBins
// equal steps of the logit gives the steps in which the limits fall, and the
// tokens of those steps are listed and sorted. The draw goes by index, so the
// kept weights are summed by segments of the row, and the segment that the
// draw falls into is gone through.
//
// One workgroup does all that for a row of up to kRowMost tokens, or for each of many rows (by_rows). Other rows go over
// the whole GPU: a pass of a few operations over 131072 tokens takes one CU 3 us, their weights 14 us.
//   k_top     the largest and smallest logit
//   k_weigh   the histogram, or, for a row without a limit, the segments' sums
//   k_gather  lists the tokens of the limits' steps; the sums of those above
//   k_pick    a workgroup a row: sorts the list, finds the end, draws
// Few rows are bound by the launches, each a chain of loads, LDS passes and barriers: 1 x 32000 (top_k 50, top_p) 3.4 + 4.2 +
// 6.0 + 6.5 us; 16 x 131072 (top_p) 4.1 + 10.3 + 8.7 + 8.1, of k_weigh 5 for adding 32 histograms of a row into one. More rows:
// 64 x 131072 (mixed) 5.3 + 11.7 + 12.5 + 11.1, of which the vector instructions (a weight takes about 20) would be 12 if they
// followed each other; the rest, those chains, was not taken apart. k_row: 333 x 50257 fp32 without a limit 35 us (1.9 TB/s of
// logits, which it reads twice), its instructions 15 spread evenly, but 77 of the 256 CUs hold two rows; 1 row of 16384 9 us
// without a limit, 16 to 20 with: one CU's passes.
// Where the steps hold more than kList tokens, the limits are found by a search over the digits of a key, which needs no list:
// rows with more equal logits than that at a limit, and ordinary rows from some 10^6 tokens on. That is slow: a row by one
// workgroup, and equal logits add to one counter in turn. 50257 equal logits 0.35 ms (0.62 with both limits; 200 rows 0.39 and
// 0.66), 2^20 6 and 11 ms, 2^22 25 and 46 ms; 2^22 normal logits with top_p 11 ms.
#include "block_common.h"
#include "head_internal.h"

namespace mq {
namespace {

typedef unsigned long long u64;

constexpr double kOne = 1099511627776.0;   // 2^40, the weight of the largest logit
constexpr float kReach = 28.5f;            // exp(-28.5) < 2^-41: no weight beyond
constexpr int kBins = 2048;
constexpr int kList = 2048;                // tokens that a workgroup sorts
constexpr int kFewest = 1024;              // a top_k up to this is listed whole, and needs no masses
constexpr int kGroup = 64 * kGroupWaves;   // k_top, k_weigh, k_gather
constexpr int kPick = 256;                 // k_pick: what runs once costs each wave of a SIMD its issue slots
constexpr int kRow = 512;                  // k_row
constexpr int64_t kRowsAtOnce = 1024;      // rows that share the workspace

// Eight logits as they lie, asked for and not waited for; -Inf where the row has ended.
template <typename T>
struct Eight {
  typedef T raw_t __attribute__((ext_vector_type(8)));
  typedef T any_t __attribute__((ext_vector_type(8), aligned(sizeof(T))));
  raw_t q;
  __device__ __forceinline__ void ask(const T* p, int left) {
    if (left >= 8) {
      q = *reinterpret_cast<const any_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = i < left ? p[i] : (T)-__builtin_inff();
    }
  }
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)q[i];
  }
};

// f(v, at, s) of the wave's pieces s = first, first + step .. < end of 512 tokens each, 8 a lane. Four are asked for before
// the first is used: a wave that waits for each by itself spends its time on that (256 rows of 50257: 24.3 us, so 23.6).
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const T* row, int vocab, int first, int end, int step, F&& f) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int s0 = first; s0 < end; s0 += 4 * step) {
    Eight<T> q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * step;
      if (s < end) q[u].ask(row + 512 * s + 8 * lane, vocab - 512 * s - 8 * lane);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u * step;
      if (s < end) {
        float v[8];
        q[u].get(v);
        f(v, 512 * s + 8 * lane, s);
      }
    }
  }
}

// A whole number that orders as the logits do (both zeros are one).
__device__ __forceinline__ uint32_t key_of(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __builtin_bit_cast(float, key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// The place of a token in its row's order: smaller comes first.
__device__ __forceinline__ u64 place_of(float l, int token) { return ((u64)~key_of(l) << 32) | (uint32_t)token; }
__device__ __forceinline__ float logit_at(u64 place) { return logit_of(~(uint32_t)(place >> 32)); }

// a b + c, c from scalar registers: a constant there needs no copy for each use.
__device__ __forceinline__ double fma_c(double a, double b, double c) {
  double d;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
  return d;
}

// rint(2^40 exp((l - top) / t)). With y = 256 (l - top) / (t ln 2) = n + r, n whole, the power is 2^(n / 256) 2^(r / 256):
// the first from a table of 256 and an exponent, the second the series of exp to the fourth power (the rest is under 2^-54,
// |r| <= 1/2). Adding 2^52 leaves the whole number in the low bits. No branch, so that a thread's eight run side by side:
// each by itself is a chain of 13 dependent fp64 steps. What lies beyond 2^-43 of the largest counts as that far, and gives
// 0. (With a table of 32 and the sixth power, the constants copied: 64 x 131072 51 us, so 49.)
constexpr int kTable = 256;
constexpr u64 kAbove = 0x4330000000000000ull;      // the bits of 2^52
struct Weigher {
  double top, scale;
  const double* table;     // 2^(40 + i / 256), in LDS
  // with the bits of 2^52 above it
  __device__ __forceinline__ u64 raw(float l) const {
    const double y = fmax(((double)l - top) * scale, -43.0 * kTable);
    const double n = rint(y), r = y - n;
    constexpr double c = 0.6931471805599453 / kTable;
    double p = fma_c(r, c * c * c * c / 24.0, c * c * c / 6.0);
    p = fma_c(p, r, c * c / 2.0);
    p = fma_c(p, r, c);
    p = fma(p, r, 1.0);
    const int k = (int)n;
    const double w = ldexp(p * table[k & (kTable - 1)], k >> 8) + 4503599627370496.0;
    return __builtin_bit_cast(u64, w);
  }
  __device__ __forceinline__ u64 operator()(float l) const { return raw(l) & 0xFFFFFFFFFFFFFull; }
};
// Fills the table; the caller's next barrier publishes it.
__device__ __forceinline__ void fill_table(double* table) {
  if (threadIdx.x < kTable) table[threadIdx.x] = kOne * exp2((double)threadIdx.x / kTable);
}

// floor(f total), f in 0 .. 1 taken to 31 bits, at most `most` steps of 2^-31; total < 2^62.
__device__ __forceinline__ u64 share(float f, u64 total, u64 most) {
  const u64 n = min((u64)((double)fminf(fmaxf(f, 0.0f), 1.0f) * 2147483648.0), most);
  return n * (total >> 31) + ((n * (total & 0x7FFFFFFFull)) >> 31);
}

// Reductions and scans over the 64 lanes by data-parallel moves (rows of 16 lanes, then across): 6 steps of a few cycles,
// where exchanges through LDS take a hundred each. `old` is what a lane without a source gets.
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int old, int v) {
  return __builtin_amdgcn_update_dpp(old, v, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 moved64(u64 old, u64 v) {
  const uint32_t lo = (uint32_t)moved<CTRL, ROWS>((int)(uint32_t)old, (int)(uint32_t)v);
  const uint32_t hi = (uint32_t)moved<CTRL, ROWS>((int)(uint32_t)(old >> 32), (int)(uint32_t)(v >> 32));
  return ((u64)hi << 32) | lo;
}
// The sum over the lanes before this one and itself.
__device__ __forceinline__ u64 scan64(u64 v) {
  v += moved64<0x111, 0xF>(0, v);
  v += moved64<0x112, 0xF>(0, v);
  v += moved64<0x114, 0xF>(0, v);
  v += moved64<0x118, 0xF>(0, v);
  v += moved64<0x142, 0xA>(0, v);
  v += moved64<0x143, 0xC>(0, v);
  return v;
}
__device__ __forceinline__ u64 last_lane(u64 v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 sum64(u64 v) { return last_lane(scan64(v)); }
// The smallest of the lanes.
__device__ __forceinline__ int least64(int v) {
  constexpr int top = 0x7FFFFFFF;
  v = min(v, moved<0x111, 0xF>(top, v));
  v = min(v, moved<0x112, 0xF>(top, v));
  v = min(v, moved<0x114, 0xF>(top, v));
  v = min(v, moved<0x118, 0xF>(top, v));
  v = min(v, moved<0x142, 0xA>(top, v));
  v = min(v, moved<0x143, 0xC>(top, v));
  return __builtin_amdgcn_readlane(v, 63);
}
__device__ __forceinline__ float least64(float v) {
  const int inf = __builtin_bit_cast(int, __builtin_inff());
  auto step = [&](int m) { v = fminf(v, __builtin_bit_cast(float, m)); };
  step(moved<0x111, 0xF>(inf, __builtin_bit_cast(int, v)));
  step(moved<0x112, 0xF>(inf, __builtin_bit_cast(int, v)));
  step(moved<0x114, 0xF>(inf, __builtin_bit_cast(int, v)));
  step(moved<0x118, 0xF>(inf, __builtin_bit_cast(int, v)));
  step(moved<0x142, 0xA>(inf, __builtin_bit_cast(int, v)));
  step(moved<0x143, 0xC>(inf, __builtin_bit_cast(int, v)));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

// The sum over the threads before this one and itself, and that of all; lds: WAVES words.
template <int WAVES>
__device__ __forceinline__ u64 scan_group(u64 v, u64* lds, u64* all) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const u64 s = scan64(v);
  __syncthreads();
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  const u64 w = lane < WAVES ? lds[lane] : 0;
  *all = sum64(w);
  return s + sum64(lane < wave ? w : 0);
}

// What a part of a row, or the row, has: its largest logit and the first place of it (of the eight tokens that hold it), its
// smallest above -Inf, and whether there is a NaN.
struct Range {
  float top, low;
  int first, bad;
};
__device__ __forceinline__ Range no_range() { return {-__builtin_inff(), __builtin_inff(), 0x7FFFFFFF, 0}; }
__device__ __forceinline__ Range join64(Range a) {
  Range g;
  g.top = -least64(-a.top);
  g.low = least64(a.low);
  g.first = least64(a.top == g.top ? a.first : 0x7FFFFFFF);
  g.bad = __any(a.bad);
  return g;
}
// The joined range of n parts, one a lane (n <= 64): every wave by itself.
__device__ __forceinline__ Range join_parts(const Range* p, int n) {
  Range a = no_range();
  if ((int)(threadIdx.x & 63) < n) a = p[threadIdx.x & 63];
  return join64(a);
}
// One instruction each; fmaxf of loaded values costs another to quiet each, which rows with a NaN do not need.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "v"(c));
  return d;
}
// By eights: `first` is where the eight tokens begin that hold the largest (token by token 17 instructions each, so 5: k_row of
// 333 x 50257 38.7 us, so 35.4; k_top of 64 x 131072 6.7 and 5.3).
__device__ __forceinline__ void look8(Range& a, const float* v, int at) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) a.bad |= __builtin_isunordered(v[i], v[i + 1]);
  const float top = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[7]));
  if (top > a.top) {
    a.top = top;
    a.first = at;
  }
  float low = min3(min3(v[0], v[1], v[2]), min3(v[3], v[4], v[5]), min3(v[6], v[7], v[7]));
  if (low == -__builtin_inff()) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[i] > -__builtin_inff() ? v[i] : __builtin_inff();
    low = min3(min3(w[0], w[1], w[2]), min3(w[3], w[4], w[5]), min3(w[6], w[7], w[7]));
  }
  a.low = min3(a.low, low, low);
}

// A row's settings, and what follows from them and its range.
struct Row {
  float top_p, u;
  int top_k;
  bool bad, greedy, has_k, has_p;
  bool listed_whole;   // a small top_k
  u64 least;           // the smallest weight that min_p lets in
  float step;          // steps of the histogram two units of the logit
  float top;
  Weigher weight;
};
__device__ __forceinline__ Row row_of(const mq_sample_args& a, int64_t r, const Range& g, const double* table) {
  Row x;
  // a setting that is not given reads u in its place, so that all five are on their way at once
  const float t_ = unwritten((a.temperature ? a.temperature : a.u) + r), top_p_ = unwritten((a.top_p ? a.top_p : a.u) + r),
              min_p_ = unwritten((a.min_p ? a.min_p : a.u) + r);
  const int top_k_ = unwritten((a.top_k ? a.top_k : reinterpret_cast<const int32_t*>(a.u)) + r);
  x.u = unwritten(a.u + r);
  const float t = a.temperature ? t_ : 1.0f, min_p = a.min_p ? min_p_ : 0.0f;
  x.top_k = a.top_k ? top_k_ : 0;
  x.top_p = a.top_p ? top_p_ : 1.0f;
  x.bad = g.bad || !(g.top > -__builtin_inff()) || !(g.top < __builtin_inff()) || !(t >= 0.0f) || !(t < __builtin_inff());
  x.greedy = t == 0.0f;
  if (!x.greedy) x.bad |= x.top_p != x.top_p || min_p != min_p || x.u != x.u;
  x.has_k = x.top_k > 0 && x.top_k < a.vocab;
  x.has_p = x.top_p < 1.0f;
  x.listed_whole = x.has_k && x.top_k <= kFewest;
  x.least = min_p > 0.0f ? (u64)ceil(fmin((double)min_p, 1.0) * kOne) : 0ull;
  x.top = g.top;
  x.step = ((float)kBins - 0.01f) / fmaxf(fminf(0.5f * kReach * t, 0.5f * g.top - 0.5f * g.low), 1e-30f);
  x.weight = {(double)g.top, kTable / ((double)t * 0.6931471805599453), table};
  return x;
}
// The step of a logit: it never falls as the logit does, so a prefix of the steps is a prefix of the order. kBins for one
// without a weight: -Inf, or further from the top than the reach. (Halves: the difference of two logits may pass fp32's
// range.)
__device__ __forceinline__ int bin_of(const Row& x, float l) {
  return (int)fminf(fmaf(l, -0.5f, 0.5f * x.top) * x.step, (float)kBins);
}

__device__ __forceinline__ void put(const mq_sample_args& a, int64_t r, int token, float logprob) {
  a.token[r] = token;
  if (a.logprob) a.logprob[r] = logprob;
}
// Rows that have no draw: the first largest logit, or none.
template <typename T>
__device__ __forceinline__ bool without_draw(const mq_sample_args& a, int64_t r, const Row& x, const Range& g, const T* row) {
  if (!x.bad && !x.greedy) return false;
  if (threadIdx.x == 0) {
    int token = -1;
    if (!x.bad)
      for (token = g.first; (float)row[token] != g.top;) ++token;      // among eight: it is there
    put(a, r, token, x.bad ? __builtin_nanf("") : 0.0f);
  }
  return true;
}

// Adds a thread's eight tokens to the histogram: counts for a limit by count, masses for one by mass.
__device__ __forceinline__ void add8(const Row& x, const float* v, u64* mass, uint32_t* count) {
  int b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = bin_of(x, v[i]);
  if (x.has_k) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (b[i] < kBins) atomicAdd(&count[b[i]], 1u);
  }
  if (x.has_p && !x.listed_whole) {
    u64 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x.weight(v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (b[i] < kBins) atomicAdd(&mass[b[i]], y[i]);
  }
}
// The sum of a thread's eight weights that min_p lets in.
__device__ __forceinline__ u64 sum8(const Row& x, const float* v) {
  u64 y[8], m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x.weight.raw(v[i]);
  if (x.least) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = y[i] >= (kAbove | x.least) ? y[i] : kAbove;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m += y[i];
  return m - 8 * kAbove;
}

// Where the limits of a row fall: the steps from p0 to p1 hold the end by mass, step k that by count (kBins: none);
// counts and masses of the steps before p0 and before k; the mass of all steps. Counts mean nothing for a row without a
// limit by count, masses for one without a limit by mass; for a small top_k the steps are all up to its own.
struct Limits {
  u64 count_p, mass_p, count_k, mass_k, total;
  int p0, p1, k;
};
__device__ __forceinline__ bool listed(const Limits& z, int bin) { return (bin >= z.p0 && bin <= z.p1) || bin == z.k; }

// Each of THREADS threads has steps that follow each other.
template <int THREADS>
__device__ __forceinline__ Limits find_limits(const Row& x, const u64* mass, const uint32_t* count, u64* lds,
                                              Limits* out) {
  constexpr int kPer = kBins / THREADS, kWaves = THREADS / 64;
  const int tid = threadIdx.x;
  const bool by_mass = x.has_p && !x.listed_whole;
  u64 m[kPer], c[kPer], ms = 0, cs = 0, total = 0, counted = 0, m0 = 0, c0 = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    m[i] = by_mass ? mass[kPer * tid + i] : 0;
    c[i] = x.has_k ? count[kPer * tid + i] : 0;
    ms += m[i];
    cs += c[i];
  }
  if (by_mass) m0 = scan_group<kWaves>(ms, lds, &total) - ms;
  if (x.has_k) c0 = scan_group<kWaves>(cs, lds, &counted) - cs;
  if (tid == 0) *out = {0, 0, counted, total, total, kBins, kBins, kBins};
  __syncthreads();
  if (x.has_k && (u64)x.top_k <= counted) {      // else all that have a weight are in
    u64 cc = c0, mm = m0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (cc < (u64)x.top_k && cc + c[i] >= (u64)x.top_k) {
        out->k = kPer * tid + i;
        out->count_k = cc;
        out->mass_k = mm;
      }
      cc += c[i];
      mm += m[i];
    }
    __syncthreads();
  }
  Limits z = *out;
  if (x.listed_whole) {
    z.p0 = 0;
    z.p1 = min(z.k, kBins - 1);
    z.count_p = z.mass_p = 0;
    return z;
  }
  if (!x.has_p) {
    z.p0 = z.p1 = z.k;
    z.count_p = z.count_k;
    return z;
  }
  // the sum of the first top_k lies between these two, and so does what the prefix has to reach
  const u64 low = max(1ull, share(x.top_p, z.mass_k, 1ull << 31));
  const u64 high = z.k < kBins ? max(1ull, share(x.top_p, z.mass_k + mass[z.k], 1ull << 31)) : low;
  u64 cc = c0, mm = m0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (mm < low && mm + m[i] >= low) {
      out->p0 = kPer * tid + i;
      out->count_p = cc;
      out->mass_p = mm;
    }
    if (mm < high && mm + m[i] >= high) out->p1 = kPer * tid + i;
    cc += c[i];
    mm += m[i];
  }
  __syncthreads();
  return *out;
}

// A thread's eight tokens: the weights of those above the limits' steps are added, those in them go to a list in LDS (only
// the first kList of them; `fill` counts all). Where no lane has one above, no weight is computed.
__device__ __forceinline__ u64 gather8(const Row& x, const Limits& z, const float* v, int at, uint32_t* fill, u64* list) {
  bool above = false;
  int b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    b[i] = bin_of(x, v[i]);
    above |= b[i] < z.p0;
    if (b[i] < kBins && listed(z, b[i])) {
      const uint32_t n = atomicAdd(fill, 1u);
      if (n < kList) list[n] = place_of(v[i], at + i);
    }
  }
  u64 m = 0;
  if (__any(above)) {
    u64 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x.weight(v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) m += b[i] < z.p0 && y[i] >= x.least ? y[i] : 0;
  }
  return m;
}

// ------------------------------------------------------------- one workgroup
struct Lds {
  u64 mass[kBins];
  uint32_t count[kBins];
  u64 place[kList];
  u64 seg[kMostSegs];
  uint32_t ties[kMostSegs];
  u64 scan[kRow / 64];
  Range range[kRow / 64];
  double table[kTable];
  Limits limits;
  u64 a, b;
  uint32_t fill;
  int i, n1;
};

// The n places in order. Few: a thread counts those before its own. More: the steps that they come from are cut again, into
// as many equal parts as kBins allows; the places are put down by parts, and then each in its part, by counting those of it
// before it (64 rows of up to 700 places: k_pick 16.4 us by counting among all up to 512 and a network beyond, so 10.9; 16
// rows of some 200: 8.1 us by counting, 9.6 by parts). Where a part holds more than kEqual (equal logits), a network sorts
// them all.
constexpr int kFew = 256;
constexpr uint32_t kEqual = 256;
template <int THREADS>
__device__ __forceinline__ void sort_places(Lds& s, const Row& x, const Limits& z, int n) {
  constexpr int kPer = kList / THREADS, kCounts = kBins / THREADS;
  const int tid = threadIdx.x;
  u64* const p = s.place;
  if (n <= kFew) {
    const u64 mine = tid < n ? p[tid] : ~0ull;
    int at = 0;
    if ((tid & ~63) < n) {
#pragma unroll 8
      for (int e = 0; e < n; ++e) at += p[e] < mine;
    }
    __syncthreads();
    if (tid < n) p[at] = mine;
    __syncthreads();
    return;
  }
  const bool gap = z.k > z.p1 && z.k < kBins;
  const int steps = z.p1 - z.p0 + 1, per = kBins / (steps + gap);
  auto part_of = [&](u64 place) {
    const float t = fmaf(logit_at(place), -0.5f, 0.5f * x.top) * x.step;
    const int b = (int)t;
    return (b <= z.p1 ? b - z.p0 : steps) * per + min((int)((t - (float)b) * (float)per), per - 1);
  };
#pragma unroll
  for (int i = 0; i < kCounts; ++i) s.count[THREADS * i + tid] = 0;
  __syncthreads();
  u64 mine[kPer];
  uint32_t slot[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = THREADS * i + tid;
    if (e < n) {
      mine[i] = p[e];
      slot[i] = atomicAdd(&s.count[part_of(mine[i])], 1u);
    }
  }
  __syncthreads();
  uint32_t c[kCounts], sum = 0, most = 0;
#pragma unroll
  for (int i = 0; i < kCounts; ++i) {
    c[i] = s.count[kCounts * tid + i];
    sum += c[i];
    most = max(most, c[i]);
  }
  u64 all;
  uint32_t before = (uint32_t)scan_group<THREADS / 64>(sum, s.scan, &all) - sum;
  if (!__syncthreads_or(most > kEqual)) {
#pragma unroll
    for (int i = 0; i < kCounts; ++i) {
      s.count[kCounts * tid + i] = before;
      before += c[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (THREADS * i + tid < n) p[s.count[part_of(mine[i])] + slot[i]] = mine[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = THREADS * i + tid;
      if (e < n) {
        mine[i] = p[e];
        const int part = part_of(mine[i]), end = part + 1 < kBins ? (int)s.count[part + 1] : n;
        slot[i] = s.count[part];
        for (int o = (int)slot[i]; o < end; ++o) slot[i] += p[o] < mine[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (THREADS * i + tid < n) p[slot[i]] = mine[i];
    __syncthreads();
    return;
  }
  // Pairs in a network: a wave's 64 pairs are 128 places that follow each other while partners are up to 64 apart, and
  // those steps need the wave alone, and no barrier.
  int n2 = 2 * (int)kEqual;
  while (n2 < n) n2 <<= 1;
  for (int e = n + tid; e < n2; e += THREADS) p[e] = ~0ull;
  bool alone = false;        // whether the last step was the wave's own
#pragma unroll 1
  for (int k = 2; k <= n2; k <<= 1) {
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      if (alone && j <= 64) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      } else {
        __syncthreads();
      }
      alone = j <= 64;
#pragma unroll 1
      for (int e = tid; e < n2 / 2; e += THREADS) {
        const int i = ((e & ~(j - 1)) << 1) | (e & (j - 1)), o = i | j;
        const u64 a = p[i], b = p[o];
        if ((a > b) == ((i & k) == 0)) {
          p[i] = b;
          p[o] = a;
        }
      }
    }
  }
  __syncthreads();
}

// Sorts the n listed places, finds the end of what is kept among them and adds the weights of those that are in to their
// segments' sums. Gives the last place that is in (there is one: the first token at which a limit by mass looks has less
// than that before it).
template <int THREADS>
__device__ __forceinline__ u64 end_of_list(Lds& s, const Row& x, const Limits& z, int n, int span) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    s.i = 0;
    s.n1 = 0;
  }
  sort_places<THREADS>(s, x, z, n);
  // The first n1 are the steps from p0 to p1; the others, behind a gap, step k. Sums of the weights before each.
  const bool gap = z.k > z.p1 && z.k < kBins;
  u64 sum = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < n; e0 += THREADS) {
    const int e = e0 + tid;
    const float l = e < n ? logit_at(s.place[e]) : -__builtin_inff();
    const u64 w = x.weight(l);
    u64 all;
    const u64 with = scan_group<THREADS / 64>(w, s.scan, &all);
    if (e < n) s.mass[e] = sum + with - w;
    if (gap && bin_of(x, l) <= z.p1) atomicAdd(&s.n1, 1);
    sum += all;
  }
  __syncthreads();
  const int n1 = gap ? s.n1 : n;
  const u64 first = n1 < n ? s.mass[n1] : sum;
  auto count = [&](int e) { return e < n1 ? z.count_p + e : z.count_k + (e - n1); };                        // tokens before it
  auto mass = [&](int e) { return e < n1 ? z.mass_p + s.mass[e] : z.mass_k + (s.mass[e] - first); };        // and their weight
  u64 need = ~0ull;
  if (x.has_p) {
    u64 total = x.listed_whole ? sum : z.total;          // of the first top_k
    if (z.k < kBins) {
      const u64 k = (u64)x.top_k - 1;                    // their last one
      const int e = k < z.count_p + n1 ? (int)(k - z.count_p) : n1 + (int)(k - z.count_k);
      total = mass(e) + x.weight(logit_at(s.place[e]));
    }
    need = max(1ull, share(x.top_p, total, 1ull << 31));
  }
  int last = 0;            // tokens of the list that are in: they are its first ones
#pragma unroll 1
  for (int e = tid; e < n; e += THREADS) {
    if ((!x.has_k || count(e) < (u64)x.top_k) && (!x.has_p || mass(e) < need)) {
      last = e + 1;
      const u64 w = x.weight(logit_at(s.place[e]));
      if (w >= x.least) atomicAdd(&s.seg[(uint32_t)s.place[e] / (uint32_t)span], w);
    }
  }
  if (last) atomicMax(&s.i, last);
  __syncthreads();
  return s.place[s.i - 1];
}

// The segment that the draw falls into (of `segs` sums in LDS), what lies before it and the sum of all.
struct Drawn {
  int seg;
  u64 before, target, total;
};
template <int THREADS>
__device__ __forceinline__ Drawn draw_segment(Lds& s, int segs, float u) {
  constexpr int kPer = kMostSegs / THREADS;
  const int tid = threadIdx.x;
  u64 m[kPer], sum = 0, total;
#pragma unroll
  for (int i = 0; i < kPer; ++i) sum += m[i] = kPer * tid + i < segs ? s.seg[kPer * tid + i] : 0;
  u64 c = scan_group<THREADS / 64>(sum, s.scan, &total) - sum;
  const u64 target = share(u, total, 0x7FFFFFFFull);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (c <= target && c + m[i] > target) {
      s.i = kPer * tid + i;
      s.a = c;
    }
    c += m[i];
  }
  __syncthreads();
  return {s.i, s.a, target, total};
}

// One of a thread's eight tokens, if the running sum passes the target in them (c: what lies before them).
__device__ __forceinline__ void draw8(const mq_sample_args& a, int64_t r, const u64* y, u64 m, u64 c, int at,
                                      const Drawn& d) {
  if (c > d.target || c + m <= d.target) return;
  int token = at;
  u64 w = y[0];
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    c += y[i];
    if (c <= d.target) {
      token = at + i + 1;
      w = y[i + 1];
    }
  }
  put(a, r, token, (float)log((double)w / (double)d.total));
}

// What a token adds where the places up to `end` are in.
__device__ __forceinline__ u64 kept(const Row& x, u64 end, float l, int token) {
  const u64 y = x.weight(l);
  return place_of(l, token) <= end && y >= x.least ? y : 0;
}

// Goes through the segment that the draw falls into.
template <int THREADS, typename T>
__device__ __forceinline__ void draw_token(Lds& s, const mq_sample_args& a, int64_t r, const Row& x, u64 end,
                                           const T* row, const Drawn& d, int span) {
  const int vocab = (int)a.vocab, stop = min(vocab, (d.seg + 1) * span);
  u64 run = d.before;
#pragma unroll 1
  for (int at0 = d.seg * span; at0 < stop; at0 += 8 * THREADS) {
    const int at = at0 + 8 * (int)threadIdx.x;
    u64 y[8] = {}, m = 0;
    if (at < stop) {
      Eight<T> q;
      float v[8];
      q.ask(row + at, vocab - at);
      q.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) m += y[i] = kept(x, end, v[i], at + i);
    }
    u64 all;
    draw8(a, r, y, m, run + scan_group<THREADS / 64>(m, s.scan, &all) - m, at, d);
    run += all;
    if (run > d.target) return;
  }
}

// The pieces of a segment.
template <typename T, typename F>
__device__ __forceinline__ void each_of_segment(const T* row, int vocab, int seg, int span, F&& f) {
  each_piece(row, vocab, seg * (span / 512), min((vocab + 511) / 512, (seg + 1) * (span / 512)), 1, f);
}

// The slow way: the limits by a search over the digits of the key, each a pass over the row. Needs no list, so it takes
// rows of any number of equal logits. A prefix is all larger keys and `ties` tokens of this one.
struct Cut {
  uint32_t key;
  u64 ties;
};

template <int THREADS, bool BY_MASS, typename T>
__device__ __forceinline__ Cut find_cut(Lds& sh, const Row& x, const T* row, int vocab, u64 need, u64* mass_in) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  uint32_t prefix = 0;
  u64 before = 0, before_mass = 0;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {      // digits of 11, 11 and 10 bits
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    const uint32_t mask = level == 2 ? 1023u : 2047u;
    for (int b = tid; b < kBins; b += THREADS) {
      sh.mass[b] = 0;
      sh.count[b] = 0;
    }
    __syncthreads();
    for (int at = 512 * wave + 8 * lane; at < vocab; at += 8 * THREADS) {
      Eight<T> q;
      float v[8];
      q.ask(row + at, vocab - at);
      q.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(v[i]);
        if (at + i < vocab && (level == 0 || (k >> (level == 1 ? 21 : 10)) == prefix)) {
          atomicAdd(&sh.count[(k >> shift) & mask], 1u);
          const u64 y = x.weight(v[i]);
          if (y) atomicAdd(&sh.mass[(k >> shift) & mask], y);
        }
      }
    }
    __syncthreads();
    if (wave == 0) {      // 32 bins a lane, from the largest on
      u64 c = 0, m = 0;
#pragma unroll 1
      for (int i = 0; i < 32; ++i) {
        const int b = kBins - 1 - (32 * lane + i);
        c += sh.count[b];
        m += sh.mass[b];
      }
      u64 c0 = before + scan64(c) - c, m0 = before_mass + scan64(m) - m;
      const u64 have = BY_MASS ? m0 : c0, then = have + (BY_MASS ? m : c);
      if (have < need && then >= need) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
          const int b = kBins - 1 - (32 * lane + i);
          const u64 c1 = c0 + sh.count[b], m1 = m0 + sh.mass[b];
          if ((BY_MASS ? m1 : c1) >= need) {
            sh.i = b;
            sh.a = c0;
            sh.b = m0;
            break;
          }
          c0 = c1;
          m0 = m1;
        }
      }
    }
    __syncthreads();
    prefix = (prefix << (level == 2 ? 10 : 11)) | (uint32_t)sh.i;
    before = sh.a;
    before_mass = sh.b;
    __syncthreads();
  }
  const u64 y = x.weight(logit_of(prefix));
  Cut cut;
  cut.key = prefix;
  cut.ties = BY_MASS ? (need - before_mass + y - 1) / y : need - before;
  *mass_in = before_mass + cut.ties * y;
  return cut;
}

template <int THREADS, typename T>
__device__ __forceinline__ void pick_by_digits(const mq_sample_args& a, int64_t r, const Row& x, const T* row, u64 total,
                                            int segs, int span, Lds& sh) {
  const int tid = threadIdx.x, wave = tid >> 6, vocab = (int)a.vocab;
  Cut cut{0u, ~0ull};         // the whole row
  u64 mass = total;
  if (x.has_k) cut = find_cut<THREADS, false>(sh, x, row, vocab, (u64)x.top_k, &mass);
  if (x.has_p) {
    const u64 need = max(1ull, share(x.top_p, mass, 1ull << 31));
    const Cut c = find_cut<THREADS, true>(sh, x, row, vocab, need, &mass);
    if (c.key > cut.key || (c.key == cut.key && c.ties < cut.ties)) cut = c;
  }
  const u64 tie = x.weight(logit_of(cut.key));
  const bool ties_in = tie >= x.least;
  // the segments' sums above the cut, and their ties
  for (int s = wave; s < segs; s += THREADS / 64) {
    u64 m = 0, n = 0;
    each_of_segment(row, vocab, s, span, [&](const float* v, int at, int) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(v[i]);
        if (k > cut.key) {
          const u64 y = x.weight(v[i]);
          if (y >= x.least) m += y;
        } else if (k == cut.key && at + i < vocab) {
          n += 1;
        }
      }
    });
    m = sum64(m);
    n = sum64(n);
    if ((tid & 63) == 0) {
      sh.seg[s] = m;
      sh.ties[s] = (uint32_t)n;
    }
  }
  __syncthreads();
  constexpr int kPer = kMostSegs / THREADS;
  u64 all, n = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += kPer * tid + i < segs ? sh.ties[kPer * tid + i] : 0;
  u64 before[kPer];
  before[0] = scan_group<THREADS / 64>(n, sh.scan, &all) - n;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * tid + i;
    if (e >= segs) continue;
    const u64 k = sh.ties[e], n_in = before[i] >= cut.ties ? 0 : min(k, cut.ties - before[i]);
    if (ties_in) sh.seg[e] += n_in * tie;
    if (i + 1 < kPer) before[i + 1] = before[i] + k;
  }
  __syncthreads();
  const Drawn d = draw_segment<THREADS>(sh, segs, x.u);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (kPer * tid + i == d.seg) sh.b = before[i];
  __syncthreads();
  // Ties count on along the segment.
  u64 run = d.before, ties = sh.b;
  const int stop = min(vocab, (d.seg + 1) * span);
  for (int at0 = d.seg * span; at0 < stop; at0 += 8 * THREADS) {
    const int at = at0 + 8 * tid;
    float v[8] = {};
    u64 y[8] = {}, m = 0, k = 0;
    if (at < stop) {
      Eight<T> q;
      q.ask(row + at, vocab - at);
      q.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) k += key_of(v[i]) == cut.key && at + i < vocab;
    }
    u64 k_all, m_all;
    u64 rank = ties + scan_group<THREADS / 64>(k, sh.scan, &k_all) - k;
    if (at < stop) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t key = key_of(v[i]);
        if (key > cut.key) {
          y[i] = x.weight(v[i]);
          if (y[i] < x.least) y[i] = 0;
        } else if (key == cut.key && at + i < vocab) {
          if (rank < cut.ties && ties_in) y[i] = tie;
          ++rank;
        }
        m += y[i];
      }
    }
    draw8(a, r, y, m, run + scan_group<THREADS / 64>(m, sh.scan, &m_all) - m, at, d);
    run += m_all;
    ties += k_all;
    if (run > d.target) return;
  }
}

// A row by a workgroup. The loops over it stay loops: what runs once is paid for by the fetch of its instructions.
template <typename T>
__global__ __launch_bounds__(kRow) void k_row(mq_sample_args a, int segs) {
  __shared__ Lds s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, vocab = (int)a.vocab;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  fill_table(s.table);
  for (int b = tid; b < kBins; b += kRow) {
    s.mass[b] = 0;
    s.count[b] = 0;
  }
  if (tid == 0) s.fill = 0;
  auto each = [&](auto&& f) { each_piece(row, vocab, wave, segs, kRow / 64, f); };
  Range g = no_range();
  each([&](const float* v, int at, int) { look8(g, v, at); });
  g = join64(g);
  if (lane == 0) s.range[wave] = g;
  __syncthreads();
  g = join_parts(s.range, kRow / 64);
  const Row x = row_of(a, r, g, s.table);
  if (without_draw(a, r, x, g, row)) return;
  auto put_sum = [&](u64 m, int seg) {
    m = sum64(m);
    if (lane == 0) s.seg[seg] = m;
  };
  u64 end = ~0ull;
  if (x.has_k || x.has_p) {
    each([&](const float* v, int, int) { add8(x, v, s.mass, s.count); });
    __syncthreads();
    const Limits z = find_limits<kRow>(x, s.mass, s.count, s.scan, &s.limits);
    each([&](const float* v, int at, int seg) { put_sum(gather8(x, z, v, at, &s.fill, s.place), seg); });
    __syncthreads();
    const uint32_t n = s.fill;
    if (n > (uint32_t)kList) {
      pick_by_digits<kRow>(a, r, x, row, z.total, segs, 512, s);
      return;
    }
    if (n > 0) end = end_of_list<kRow>(s, x, z, (int)n, 512);
  } else {
    each([&](const float* v, int, int seg) { put_sum(sum8(x, v), seg); });
  }
  __syncthreads();
  draw_token<kRow>(s, a, r, x, end, row, draw_segment<kRow>(s, segs, x.u), 512);
}

// ------------------------------------------------------------ the whole GPU
struct Work {
  u64* mass;        // [rows, kBins]
  uint32_t* count;  // [rows, kBins]
  u64* list;        // [rows, kList]
  uint32_t* fill;   // [rows]
  Limits* limits;   // [rows]
  Range* range;     // [rows, splits]
  u64* seg;         // [rows, kGroupWaves splits]
  int splits;       // workgroups a row, of kGroupWaves segments each
  int span;         // tokens of a segment
};

template <typename T>
__global__ __launch_bounds__(kGroup) void k_top(mq_sample_args a, Work w, int limits) {
  __shared__ Range lds[kGroupWaves];
  const int64_t r = blockIdx.y;
  const int s = blockIdx.x, tid = threadIdx.x;
  if (limits) {        // the row's histogram, which the next launch adds to
    const int per = (kBins + w.splits - 1) / w.splits;
    for (int b = s * per + tid; b < min(kBins, (s + 1) * per); b += kGroup) {
      w.mass[r * kBins + b] = 0;
      w.count[r * kBins + b] = 0;
    }
    if (s == 0 && tid == 0) w.fill[r] = 0;
  }
  Range g = no_range();
  each_of_segment(static_cast<const T*>(a.logits) + r * a.stride, (int)a.vocab, kGroupWaves * s + (tid >> 6), w.span,
        [&](const float* v, int at, int) { look8(g, v, at); });
  g = join64(g);
  if ((tid & 63) == 0) lds[tid >> 6] = g;
  __syncthreads();
  g = join_parts(lds, kGroupWaves);
  if (tid == 0) w.range[r * w.splits + s] = g;
}

template <typename T>
__global__ __launch_bounds__(kGroup) void k_weigh(mq_sample_args a, Work w) {
  __shared__ u64 mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ double table[kTable];
  const int64_t r = blockIdx.y;
  const int tid = threadIdx.x, seg = kGroupWaves * blockIdx.x + (tid >> 6);
  fill_table(table);
  for (int b = tid; b < kBins; b += kGroup) {
    mass[b] = 0;
    count[b] = 0;
  }
  const Row x = row_of(a, r, join_parts(w.range + r * w.splits, w.splits), table);
  __syncthreads();
  if (x.bad || x.greedy) return;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  if (!x.has_k && !x.has_p) {
    u64 m = 0;
    each_of_segment(row, (int)a.vocab, seg, w.span, [&](const float* v, int, int) { m += sum8(x, v); });
    m = sum64(m);
    if ((tid & 63) == 0) w.seg[r * kGroupWaves * w.splits + seg] = m;
    return;
  }
  each_of_segment(row, (int)a.vocab, seg, w.span, [&](const float* v, int, int) { add8(x, v, mass, count); });
  __syncthreads();
  for (int b = tid; b < kBins; b += kGroup) {
    if (mass[b]) atomicAdd(&w.mass[r * kBins + b], mass[b]);
    if (count[b]) atomicAdd(&w.count[r * kBins + b], count[b]);
  }
}

template <typename T>
__global__ __launch_bounds__(kGroup) void k_gather(mq_sample_args a, Work w) {
  __shared__ u64 lds[kGroupWaves], list[kList];
  __shared__ Limits lds_limits;
  __shared__ double table[kTable];
  __shared__ uint32_t fill, base;
  const int64_t r = blockIdx.y;
  const int tid = threadIdx.x, seg = kGroupWaves * blockIdx.x + (tid >> 6);
  fill_table(table);
  if (tid == 0) fill = 0;
  const Row x = row_of(a, r, join_parts(w.range + r * w.splits, w.splits), table);
  if (x.bad || x.greedy || (!x.has_k && !x.has_p)) return;
  const Limits z = find_limits<kGroup>(x, w.mass + r * kBins, w.count + r * kBins, lds, &lds_limits);
  if (blockIdx.x == 0 && tid == 0) w.limits[r] = z;
  u64 m = 0;
  each_of_segment(static_cast<const T*>(a.logits) + r * a.stride, (int)a.vocab, seg, w.span,
        [&](const float* v, int at, int) { m += gather8(x, z, v, at, &fill, list); });
  m = sum64(m);
  if ((tid & 63) == 0) w.seg[r * kGroupWaves * w.splits + seg] = m;
  // the workgroup's list joins the row's; their order there is any: k_pick sorts them
  __syncthreads();
  const uint32_t n = fill;
  if (n == 0) return;
  if (tid == 0) base = atomicAdd(&w.fill[r], n);
  __syncthreads();
  for (uint32_t e = tid; e < n && base + e < (uint32_t)kList; e += kGroup) w.list[r * kList + base + e] = list[e];
}

template <typename T>
__global__ __launch_bounds__(kPick) void k_pick(mq_sample_args a, Work w) {
  __shared__ Lds s;
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, segs = kGroupWaves * w.splits;
  const T* row = static_cast<const T*>(a.logits) + r * a.stride;
  fill_table(s.table);
  // all that may be needed is asked for at once (what a row without limits never wrote is not looked at)
  const Limits z = w.limits[r];
  const uint32_t n = w.fill[r];
  const u64 sum = tid < segs ? w.seg[r * segs + tid] : 0, place = w.list[r * kList + tid];
  const Range g = join_parts(w.range + r * w.splits, w.splits);
  const Row x = row_of(a, r, g, s.table);
  if (without_draw(a, r, x, g, row)) return;
  if (tid < segs) s.seg[tid] = sum;
  for (int e = kPick + tid; e < segs; e += kPick) s.seg[e] = w.seg[r * segs + e];
  u64 end = ~0ull;                         // the last place that is in
  if (x.has_k || x.has_p) {
    if (n > (uint32_t)kList) {
      __syncthreads();
      pick_by_digits<kPick>(a, r, x, row, z.total, segs, w.span, s);
      return;
    }
    if (tid < (int)n) s.place[tid] = place;
    for (int e = kPick + tid; e < (int)n; e += kPick) s.place[e] = w.list[r * kList + e];
    __syncthreads();
    if (n > 0) end = end_of_list<kPick>(s, x, z, (int)n, w.span);
  }
  __syncthreads();
  const Drawn d = draw_segment<kPick>(s, segs, x.u);
  draw_token<kPick>(s, a, r, x, end, row, d, w.span);
}

// ------------------------------------------------------------------- the host
size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

// The workspace of so many rows at once; base may be null, for its size alone.
Work lay_out(char* base, int64_t rows, int64_t vocab, size_t* bytes) {
  Work w;
  split(rows, vocab, &w.splits, &w.span);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* p = base ? base + at : nullptr;
    at += up16(n);
    return p;
  };
  w.mass = reinterpret_cast<u64*>(take(rows * kBins * 8));
  w.count = reinterpret_cast<uint32_t*>(take(rows * kBins * 4));
  w.list = reinterpret_cast<u64*>(take(rows * kList * 8));
  w.fill = reinterpret_cast<uint32_t*>(take(rows * 4));
  w.limits = reinterpret_cast<Limits*>(take(rows * sizeof(Limits)));
  w.range = reinterpret_cast<Range*>(take(rows * w.splits * sizeof(Range)));
  w.seg = reinterpret_cast<u64*>(take(rows * w.splits * kGroupWaves * 8));
  if (bytes) *bytes = at;
  return w;
}

template <typename T>
hipError_t go(const mq_sample_args& a, void* ws, hipStream_t s) {
  const dim3 rows((unsigned)a.rows);
  if (by_rows(a.rows, a.vocab)) {
    k_row<T><<<rows, dim3(kRow), 0, s>>>(a, (int)((a.vocab + 511) / 512));
    return hipGetLastError();
  }
  for (int64_t r = 0; r < a.rows; r += kRowsAtOnce) {
    mq_sample_args b = a;
    b.rows = a.rows - r < kRowsAtOnce ? a.rows - r : kRowsAtOnce;
    b.logits = static_cast<const T*>(a.logits) + r * a.stride;
    if (a.temperature) b.temperature = a.temperature + r;
    if (a.top_k) b.top_k = a.top_k + r;
    if (a.top_p) b.top_p = a.top_p + r;
    if (a.min_p) b.min_p = a.min_p + r;
    b.u = a.u + r;
    b.token = a.token + r;
    if (a.logprob) b.logprob = a.logprob + r;
    const Work w = lay_out(static_cast<char*>(ws), b.rows, a.vocab, nullptr);
    const dim3 grid((unsigned)w.splits, (unsigned)b.rows);
    const bool limits = a.top_k || a.top_p;
    k_top<T><<<grid, dim3(kGroup), 0, s>>>(b, w, limits);
    k_weigh<T><<<grid, dim3(kGroup), 0, s>>>(b, w);
    if (limits) k_gather<T><<<grid, dim3(kGroup), 0, s>>>(b, w);
    k_pick<T><<<dim3((unsigned)b.rows), dim3(kPick), 0, s>>>(b, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t sample_workspace(int64_t rows, int64_t vocab, int) {
  if (rows == 0 || by_rows(rows, vocab)) return 0;
  size_t n;
  lay_out(nullptr, rows < kRowsAtOnce ? rows : kRowsAtOnce, vocab, &n);
  const int64_t rest = rows % kRowsAtOnce;      // the last rows are cut into more segments each
  if (rows > kRowsAtOnce && rest > 0) {
    size_t m;
    lay_out(nullptr, rest, vocab, &m);
    n = n > m ? n : m;
  }
  return n;
}

hipError_t launch_sample(const mq_sample_args& a, void* ws, hipStream_t s) {
  return a.logits_fp32 ? go<float>(a, ws, s) : go<_Float16>(a, ws, s);
}

}  // namespace mq
