// Attention over the 8-bit key/value cache for many query rows: prompts and
// their pieces (kv_attn.hip holds the kernel for few rows and the join).
//
// A workgroup of W waves holds 32 W rows of one kv head (row r = new token
// r / g, query head r % g, so the g heads that share the keys share the
// tile) and walks the 64-token blocks they see. A block's codes are loaded
// two blocks ahead into registers, widened once for the workgroup and laid
// into LDS as fp16; every wave multiplies them with its own 32 rows:
//   S^T = K Q^T    32x32x16 fp16 MFMA, two tiles of 32 tokens. Lane (c, f) =
//                  (l % 32, l / 32) gets row c and, with tile row R holding
//                  token 16 (R / 16) + 8 (R / 4 % 2) + 4 (R / 8 % 2) + R % 4,
//                  the tokens 16 x + 8 f + 0..7 of both halves x of the tile:
//   O^T += V^T P^T just the B operand of this product, without LDS.
// The block's scales stay in fp32: with t = (k scale) s + log2(v scale) the
// weights are p = 2^(t - m), so that O sums codes in units of 2^-m and no block
// needs its own accumulator; the softmax's sum takes p / (v scale). The
// reference m follows the running maximum only when that has grown by more
// than 2^8 (p then reaches 2^8 at most, far inside fp16), so the sums are
// rarely rescaled. p is rounded to fp16 (relative 2^-11), its sum is not.
// LDS rows are swizzled by 16-byte pieces: the 8 lanes that read together hit
// different banks.
// Bound by the matrix cores and the exponentials beside them.
#include "kv_attn_common.h"

namespace mq {
namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float16_t mfma32(half8_t a, half8_t b, float16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The larger (the sum) of lanes l and l ^ 32, in both.
__device__ __forceinline__ float max_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const u32x2_t r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r.x), __builtin_bit_cast(float, (uint32_t)r.y));
}
__device__ __forceinline__ float sum_halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const u32x2_t r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (uint32_t)r.x) + __builtin_bit_cast(float, (uint32_t)r.y);
}

constexpr float kNoMax = -1.0e30f;   // the reference before the first visible token: finite, below every score
constexpr float kSlack = 8.0f;       // how far (powers of two) the maximum may run ahead of the reference
constexpr float kZeroScale = 1.0f / (1 << 30);   // stands for the scale of values that are all zero

// The swizzle of a key row and of a value row: 16-byte piece -> place.
__device__ __forceinline__ int key_place(int token, int piece) {
  return piece ^ ((token & 3) | ((token >> 1) & 4));
}
__device__ __forceinline__ int value_place(int d, int piece) { return piece ^ (d & 7); }

template <int D, int FMT, int W>
__global__ __launch_bounds__(64 * W, 2) void k_attn_rows(AttnArgs A) {
  constexpr int THREADS = 64 * W, KS = D / 16, DT = D / 32;
  constexpr int PIECES = kKvBlock * D / 16;               // 16-byte pieces of codes of a block's keys (and values)
  constexpr int LOADS = (2 * PIECES + THREADS - 1) / THREADS;
  static_assert(2 * PIECES % THREADS == 0 && PIECES % 64 == 0, "a wave loads keys or values, not both");
  __shared__ __attribute__((aligned(16))) _Float16 lk[2][kKvBlock * D], lv[2][kKvBlock * D];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 31, f = lane >> 5;

  // workgroup -> (row tile, the last first: it sees the most; sequence; split; kv head)
  int w = (int)blockIdx.x;
  const int h = w % A.kv.hk;
  w /= A.kv.hk;
  const int split = w % A.splits;
  w /= A.splits;
  const int s = w % A.b.seqs, rt = A.row_tiles - 1 - w / A.b.seqs;
  const Seq sq = seq_of(A.b, A.kv, s);
  const int rows = sq.n * A.group, row0 = rt * 32 * W;
  if (row0 >= rows) return;
  const int len = sq.cap;

  // this lane's row
  const int r = row0 + 32 * wave + c;
  const int rr = r < rows ? r : row0;
  const int tok = rr / A.group, hh = rr % A.group;
  const int end = r >= rows ? 0 : A.causal ? max(len - sq.n + tok + 1, 0) : len;
  half8_t qf[KS];
  {
    const _Float16* qp = A.q.p + (int64_t)(sq.q0 + tok) * A.q.stride + (int64_t)(h * A.group + hh) * D;
    const bool flip = A.scale2 < 0.0f;   // a negative scale turns the queries: scores can then be compared before they are scaled
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qf[k] = *reinterpret_cast<const half8_t*>(qp + 16 * k + 8 * f);
      if (flip) qf[k] = -qf[k];
    }
  }
  const float scale2 = fabsf(A.scale2);
  // blocks the workgroup and this wave see, and the tokens that every row of the wave sees
  const int last_row = min(rows, row0 + 32 * W) - 1;
  const int group_end = A.causal ? max(len - sq.n + last_row / A.group + 1, 0) : len;
  int wave_end = end, wave_all = r < rows ? end : len;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    wave_end = max(wave_end, __shfl_xor(wave_end, d));
    wave_all = min(wave_all, __shfl_xor(wave_all, d));
  }
  wave_end = __builtin_amdgcn_readfirstlane(wave_end);
  wave_all = __builtin_amdgcn_readfirstlane(wave_all);
  const int nblk = (group_end + kKvBlock - 1) / kKvBlock;
  const int b0 = split * A.chunk, b1 = min(nblk, b0 + A.chunk);
  const int open_blk = len / kKvBlock;
  const int32_t* table = A.b.table + (int64_t)s * A.b.width;

  float16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNoMax, l = 0.0f;

  // the next block's codes, in registers
  uint4 codes[LOADS];
  const auto load = [&](int b) {
    if (b >= b1 || b == open_blk) return;
    const int id0 = table[b];
    const int64_t head = ((uint64_t)(int64_t)id0 < (uint64_t)A.kv.blocks ? (int64_t)id0 : 0) * A.kv.hk + h;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int p = tid + i * THREADS;
      const uint8_t* base = p < PIECES ? A.kv.kc : A.kv.vc;
      codes[i] = *reinterpret_cast<const uint4*>(base + head * (kKvBlock * D) + (int64_t)(p % PIECES) * 16);
    }
  };
  // lays block b into LDS buffer x
  const auto lay = [&](int b, int x) {
    if (b >= b1) return;
    if (b != open_blk) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int p = tid + i * THREADS;
        const half8_t lo = widen8<FMT>(codes[i].x, codes[i].y), hi = widen8<FMT>(codes[i].z, codes[i].w);
        if (p < PIECES) {
          const int t = p / (D / 16), piece = 2 * (p % (D / 16));
          *reinterpret_cast<half8_t*>(&lk[x][t * D + 8 * key_place(t, piece)]) = lo;
          *reinterpret_cast<half8_t*>(&lk[x][t * D + 8 * key_place(t, piece + 1)]) = hi;
        } else {
          const int q = p - PIECES, d = q / 4, piece = 2 * (q % 4);
          *reinterpret_cast<half8_t*>(&lv[x][d * kKvBlock + 8 * value_place(d, piece)]) = lo;
          *reinterpret_cast<half8_t*>(&lv[x][d * kKvBlock + 8 * value_place(d, piece + 1)]) = hi;
        }
      }
    } else {   // the open block is fp16; tokens from `left` on are not the sequence's and may be no numbers
      const int left = len - b * kKvBlock;
      const int64_t head = ((int64_t)max(sq.slot, 0) * A.kv.hk + h) * (kKvBlock * D);
      for (int p = tid; p < 2 * PIECES; p += THREADS) {
        const int t = p / (D / 8), piece = p % (D / 8);
        *reinterpret_cast<half8_t*>(&lk[x][t * D + 8 * key_place(t, piece)]) =
            *reinterpret_cast<const half8_t*>(A.kv.kt + head + 8 * p);
        const int d = p / 8, vp = p % 8;
        half8_t v = *reinterpret_cast<const half8_t*>(A.kv.vt + head + 8 * p);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * vp + i >= left) v[i] = (_Float16)0.0f;
        *reinterpret_cast<half8_t*>(&lv[x][d * kKvBlock + 8 * value_place(d, vp)]) = v;
      }
    }
  };

  if (b0 < b1) {
    load(b0);
    lay(b0, 0);
    load(b0 + 1);
  }
  __syncthreads();
  const int ktok = 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);
  for (int b = b0; b < b1; ++b) {
    const int x = (b - b0) & 1;
    lay(b + 1, x ^ 1);
    load(b + 2);
    if (b * kKvBlock < wave_end) {
      float ks, vs;
      if (b != open_blk) {
        const int id0 = table[b];
        const bool ok = (uint64_t)(int64_t)id0 < (uint64_t)A.kv.blocks;
        const int64_t head = (int64_t)(ok ? id0 : 0) * A.kv.hk + h;
        ks = ok ? A.kv.ks[head] : __builtin_nanf("");
        vs = A.kv.vs[head];
        vs = vs == 0.0f ? kZeroScale : vs;
      } else {
        ks = sq.slot >= 0 ? 1.0f : __builtin_nanf("");
        vs = 1.0f;
      }
      float16_t sc[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[t][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int token = 32 * t + ktok;
          const half8_t a = *reinterpret_cast<const half8_t*>(&lk[x][token * D + 8 * key_place(token, 2 * k + f)]);
          sc[t] = mfma32(a, qf[k], sc[t]);
        }
      }
      const float mul = ks * scale2, add = __builtin_amdgcn_logf(vs);
      const bool masked = (b + 1) * kKvBlock > wave_all;
      // sc[t][8 x2 + j] is token 32 t + 16 x2 + 8 f + j of the block
      const int left = end - b * kKvBlock - 8 * f;
      if (masked) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (32 * t + 16 * (i >> 3) + (i & 7) >= left) sc[t][i] = -INFINITY;
      }
      float top = sc[0][0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, sc[i >> 4][i & 15]);
      top = max_halves(top);
      top = top == -INFINITY ? kNoMax : fmaf(top, mul, add);
      if (__any(top > m + kSlack)) {
        const float now = fmaxf(m, top);
        const float shrink = __builtin_amdgcn_exp2f(m - now);
        m = now;
        l *= shrink;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= shrink;
      }
      const float off = add - m;
      float sum = 0.0f;
      half8_t pf[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float p = __builtin_amdgcn_exp2f(fmaf(sc[t][i], mul, off));
          if (masked && 32 * t + 16 * (i >> 3) + (i & 7) >= left) p = 0.0f;
          sum += p;
          pf[t][i >> 3][i & 7] = (_Float16)p;
        }
      l = fmaf(sum, 1.0f / vs, l);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int row = 32 * d + c;
            const half8_t a = *reinterpret_cast<const half8_t*>(
                &lv[x][row * kKvBlock + 8 * value_place(row, 4 * t + 2 * y + f)]);
            o[d] = mfma32(a, pf[t][y], o[d]);
          }
    }
    __syncthreads();
  }

  l = sum_halves(l);
  if (r >= rows) return;
  const int64_t row = (int64_t)(sq.q0 + tok) * A.hq + h * A.group + hh;
  if (A.splits == 1) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    _Float16* out = A.out.p + (int64_t)(sq.q0 + tok) * A.out.stride + (int64_t)(h * A.group + hh) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4_t v = {o[d][i] * inv, o[d][i + 1] * inv, o[d][i + 2] * inv, o[d][i + 3] * inv};
        store4(reinterpret_cast<uint16_t*>(out + 32 * d + 2 * i + 4 * f), v, 4, true);
      }
  } else {
    float* out = A.ws_o + (row * A.splits + split) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4_t*>(out + 32 * d + 2 * i + 4 * f) =
            (float4_t){o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (f == 0) A.ws_ml[row * A.splits + split] = make_float2(m, l);
  }
}

template <int D, int FMT>
void go(const AttnArgs& A, const AttnPlan& p, hipStream_t s) {
  const dim3 g((unsigned)p.groups);
  if (p.waves == 8)
    k_attn_rows<D, FMT, 8><<<g, dim3(512), 0, s>>>(A);
  else
    k_attn_rows<D, FMT, 4><<<g, dim3(256), 0, s>>>(A);
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& A, int dim, int format, const AttnPlan& p, hipStream_t s) {
  if (dim == 64) {
    if (format == MQ_KV_INT8) go<64, MQ_KV_INT8>(A, p, s); else go<64, MQ_KV_E4M3>(A, p, s);
  } else {
    if (format == MQ_KV_INT8) go<128, MQ_KV_INT8>(A, p, s); else go<128, MQ_KV_E4M3>(A, p, s);
  }
  return hipGetLastError();
}

}  // namespace mq
