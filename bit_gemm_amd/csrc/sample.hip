// A token for each row of logits from given random numbers
// (include/mosaicq_head.h, mq_sample).
//
// Weights are whole numbers of 2^-40 of the largest, so sums of them are exact
// and no order of additions, split or atomic can change a result. What is kept
// is a prefix of the tokens in the order of their logits; its end, for a count
// (top-k) or a mass (top-p), is found by a search over the digits of an
// order-preserving key, and is the pair of a key and how many of the tokens
// with that key are in.
#include "block_common.h"
#include "head_internal.h"

namespace mq {
namespace {

typedef unsigned long long u64;

constexpr double kOne = 1099511627776.0;   // 2^40, the weight of the largest logit
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSeg = 512;                  // tokens of a segment: 8 a lane
constexpr int kBins = 2048;

__device__ __forceinline__ void take8(const _Float16* p, int64_t left, float* v) {
  if (left >= 8) {
    const half8_t h = load8(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)p[i] : -__builtin_inff();
  }
}
__device__ __forceinline__ void take8(const float* p, int64_t left, float* v) {
  if (left >= 8) {
    const float4_t a = reinterpret_cast<const float4_any_t*>(p)[0], b = reinterpret_cast<const float4_any_t*>(p + 4)[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[i + 4] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : -__builtin_inff();
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

__device__ __forceinline__ u64 weight(float l, double top, double inv_t) {
  return (u64)rint(kOne * exp(((double)l - top) * inv_t));
}

// floor(f total), f in 0 .. 1 taken to 31 bits, at most `most` steps of 2^-31; total < 2^62.
__device__ __forceinline__ u64 share(float f, u64 total, u64 most) {
  const u64 n = min((u64)((double)fminf(fmaxf(f, 0.0f), 1.0f) * 2147483648.0), most);
  return n * (total >> 31) + ((n * (total & 0x7FFFFFFFull)) >> 31);
}

__device__ __forceinline__ u64 sum64(u64 v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The sum over the lanes before this one and itself.
__device__ __forceinline__ u64 scan64(u64 v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}

// Where a prefix ends: tokens with a larger key are in, and `ties` of those with this key.
struct Cut {
  uint32_t key;
  u64 ties;
};

struct Shared {
  u64 mass[kBins];
  uint32_t count[kBins];
  float top[kWaves];
  int bad[kWaves];
  int first[kWaves];
  uint32_t bin;
  u64 before;
  u64 before_mass;
};

template <typename T>
struct Row {
  const T* p;
  int vocab;
  double top, inv_t;
};

// The smallest prefix whose count (BY_MASS false) or mass reaches `need` (at most that of the whole row): its cut, and its mass.
template <typename T, bool BY_MASS>
__device__ Cut find_cut(Shared& sh, const Row<T>& row, u64 need, u64* mass) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int segs = (row.vocab + kSeg - 1) / kSeg;
  uint32_t prefix = 0;
  u64 before = 0, before_mass = 0;
  // digits of 11, 11 and 10 bits
  for (int level = 0; level < 3; ++level) {
    const int shift = level == 0 ? 21 : level == 1 ? 10 : 0;
    const uint32_t mask = level == 2 ? 1023u : 2047u;
    for (int b = tid; b < kBins; b += kThreads) {
      sh.mass[b] = 0;
      sh.count[b] = 0;
    }
    __syncthreads();
    for (int s = wave; s < segs; s += kWaves) {
      const int at = s * kSeg + 8 * lane;
      float v[8];
      take8(row.p + at, row.vocab - at, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t k = key_of(v[i]);
        if (at + i < row.vocab && (level == 0 || (k >> (level == 1 ? 21 : 10)) == prefix)) {
          atomicAdd(&sh.count[(k >> shift) & mask], 1u);
          atomicAdd(&sh.mass[(k >> shift) & mask], weight(v[i], row.top, row.inv_t));
        }
      }
    }
    __syncthreads();
    if (wave == 0) {      // 32 bins a lane, from the largest on
      u64 c = 0, m = 0;
      for (int i = 0; i < 32; ++i) {
        const int b = kBins - 1 - (32 * lane + i);
        c += sh.count[b];
        m += sh.mass[b];
      }
      const u64 cs = scan64(c), ms = scan64(m);
      u64 c0 = before + cs - c, m0 = before_mass + ms - m;
      const u64 have = BY_MASS ? m0 : c0, then = have + (BY_MASS ? m : c);
      if (have < need && then >= need) {
        for (int i = 0; i < 32; ++i) {
          const int b = kBins - 1 - (32 * lane + i);
          const u64 c1 = c0 + sh.count[b], m1 = m0 + sh.mass[b];
          if ((BY_MASS ? m1 : c1) >= need) {
            sh.bin = (uint32_t)b;
            sh.before = c0;
            sh.before_mass = m0;
            break;
          }
          c0 = c1;
          m0 = m1;
        }
      }
    }
    __syncthreads();
    prefix = (prefix << (level == 2 ? 10 : 11)) | sh.bin;
    before = sh.before;
    before_mass = sh.before_mass;
    __syncthreads();
  }
  const u64 w = weight(logit_of(prefix), row.top, row.inv_t);
  Cut cut;
  cut.key = prefix;
  cut.ties = BY_MASS ? (need - before_mass + w - 1) / w : need - before;
  *mass = before_mass + cut.ties * w;
  return cut;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_sample(mq_sample_args a) {
  __shared__ Shared sh;
  extern __shared__ u64 seg_mass[];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int vocab = (int)a.vocab, segs = (vocab + kSeg - 1) / kSeg;
  uint32_t* seg_ties = reinterpret_cast<uint32_t*>(seg_mass + segs);
  Row<T> row{static_cast<const T*>(a.logits) + r * a.stride, vocab, 0.0, 1.0};
  const float t = a.temperature ? a.temperature[r] : 1.0f;

  // the largest logit and the first place of it
  float top = -__builtin_inff();
  int first = 0x7FFFFFFF, bad = 0;
  for (int s = wave; s < segs; s += kWaves) {
    const int at = s * kSeg + 8 * lane;
    float v[8];
    take8(row.p + at, vocab - at, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      bad |= !(v[i] < __builtin_inff());
      if (v[i] > top) {
        top = v[i];
        first = at + i;
      }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const float o = __shfl_xor(top, d);
    const int f = __shfl_xor(first, d);
    if (o > top || (o == top && f < first)) {
      top = o;
      first = f;
    }
    bad |= __shfl_xor(bad, d);
  }
  if (lane == 0) {
    sh.top[wave] = top;
    sh.first[wave] = first;
    sh.bad[wave] = bad;
  }
  __syncthreads();
  for (int k = 0; k < kWaves; ++k) {
    if (sh.top[k] > top || (sh.top[k] == top && sh.first[k] < first)) {
      top = sh.top[k];
      first = sh.first[k];
    }
    bad |= sh.bad[k];
  }
  const float top_p = a.top_p ? a.top_p[r] : 1.0f, min_p = a.min_p ? a.min_p[r] : 0.0f, u = a.u[r];
  const int top_k = a.top_k ? a.top_k[r] : 0;
  bad |= !(top > -__builtin_inff()) || !(t >= 0.0f) || !(t < __builtin_inff());
  if (t != 0.0f) bad |= top_p != top_p || min_p != min_p || u != u;
  if (bad || t == 0.0f) {
    if (tid == 0) {
      a.token[r] = bad ? -1 : first;
      if (a.logprob) a.logprob[r] = bad ? __builtin_nanf("") : 0.0f;
    }
    return;
  }
  row.top = (double)top;
  row.inv_t = 1.0 / (double)t;

  Cut cut{0u, ~0ull};         // the whole row
  u64 mass = 0;
  if (top_k > 0 && top_k < vocab) cut = find_cut<T, false>(sh, row, (u64)top_k, &mass);
  if (top_p < 1.0f) {
    if (mass == 0) {
      u64 m = 0;
      for (int s = wave; s < segs; s += kWaves) {
        const int at = s * kSeg + 8 * lane;
        float v[8];
        take8(row.p + at, vocab - at, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) m += weight(v[i], row.top, row.inv_t);
      }
      m = sum64(m);
      if (lane == 0) sh.mass[wave] = m;
      __syncthreads();
      for (int k = 0; k < kWaves; ++k) mass += sh.mass[k];
      __syncthreads();
    }
    const u64 need = max(1ull, share(top_p, mass, 1ull << 31));
    const Cut c = find_cut<T, true>(sh, row, need, &mass);
    if (c.key > cut.key || (c.key == cut.key && c.ties < cut.ties)) cut = c;
  }
  const double least = min_p > 0.0f ? fmin((double)min_p, 1.0) * kOne : 0.0;
  const float cut_l = logit_of(cut.key);
  const u64 w_tie = cut.ties == ~0ull ? 0ull : weight(cut_l, row.top, row.inv_t);
  const bool ties_in = (double)w_tie >= least;

  // the kept weight of each segment: above the cut, and how many ties it has
  for (int s = wave; s < segs; s += kWaves) {
    const int at = s * kSeg + 8 * lane;
    float v[8];
    take8(row.p + at, vocab - at, v);
    u64 m = 0, n = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t k = key_of(v[i]);
      if (k > cut.key) {
        const u64 w = weight(v[i], row.top, row.inv_t);
        if ((double)w >= least) m += w;
      } else if (k == cut.key && at + i < vocab) {
        n += 1;
      }
    }
    m = sum64(m);
    n = sum64(n);
    if (lane == 0) {
      seg_mass[s] = m;
      seg_ties[s] = (uint32_t)n;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  // The first wave walks the segments: twice, for the sum and for the place.
  u64 total = 0, target = 0;
  int at_seg = 0;
  u64 seg_before = 0, ties_before = 0;
  for (int pass = 0; pass < 2; ++pass) {
    u64 run = 0, ties = 0;
    for (int s0 = 0; s0 < segs; s0 += 64) {
      const int s = s0 + lane;
      const u64 n = s < segs ? seg_ties[s] : 0;
      const u64 ns = scan64(n) + ties;       // with this segment
      const u64 n_in = ns - n >= cut.ties ? 0 : min(n, cut.ties - (ns - n));
      const u64 m = (s < segs ? seg_mass[s] : 0) + (ties_in ? n_in * w_tie : 0);
      const u64 ms = scan64(m) + run;
      if (pass == 1) {
        const u64 hit = __ballot(ms > target);
        if (hit) {
          const int w = __ffsll(hit) - 1;
          at_seg = s0 + w;
          seg_before = __shfl(ms - m, w);
          ties_before = __shfl(ns - n, w);
          break;
        }
      }
      run = __shfl(ms, 63);
      ties = __shfl(ns, 63);
    }
    if (pass == 0) {
      total = run;
      target = share(u, total, 0x7FFFFFFFull);
    }
  }
  // and the token in it
  const int at = at_seg * kSeg + 8 * lane;
  float v[8];
  take8(row.p + at, vocab - at, v);
  u64 w[8], n = 0, m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) n += key_of(v[i]) == cut.key && at + i < vocab;
  u64 rank = ties_before + scan64(n) - n;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t k = key_of(v[i]);
    w[i] = 0;
    if (k > cut.key) {
      w[i] = weight(v[i], row.top, row.inv_t);
      if ((double)w[i] < least) w[i] = 0;
    } else if (k == cut.key && at + i < vocab) {
      if (rank < cut.ties && ties_in) w[i] = w_tie;
      ++rank;
    }
    m += w[i];
  }
  u64 run = seg_before + scan64(m) - m;
  int token = -1;
  u64 tw = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    run += w[i];
    if (token < 0 && run > target) {
      token = at + i;
      tw = w[i];
    }
  }
  const u64 hit = __ballot(token >= 0);
  if (hit && lane == __ffsll(hit) - 1) {
    a.token[r] = token;
    if (a.logprob) a.logprob[r] = (float)log((double)tw / (double)total);
  }
}

}  // namespace

size_t sample_workspace(int64_t rows, int64_t vocab, int fp32) { return 0; }

hipError_t launch_sample(const mq_sample_args& a, void* ws, hipStream_t s) {
  if (a.rows == 0) return hipSuccess;
  const int64_t segs = (a.vocab + kSeg - 1) / kSeg;
  const size_t lds = (size_t)segs * 12;
  const void* f = a.logits_fp32 ? reinterpret_cast<const void*>(&k_sample<float>) : reinterpret_cast<const void*>(&k_sample<_Float16>);
  if (lds > 32768) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  if (a.logits_fp32) k_sample<float><<<dim3((unsigned)a.rows), dim3(kThreads), lds, s>>>(a);
  else k_sample<_Float16><<<dim3((unsigned)a.rows), dim3(kThreads), lds, s>>>(a);
  return hipGetLastError();
}

}  // namespace mq
