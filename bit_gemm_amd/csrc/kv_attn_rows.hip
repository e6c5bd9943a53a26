// Attention over the 8-bit key/value cache for many query rows: prompts and
// their pieces (kv_attn.hip holds the kernel for few rows and the join).
//
// A workgroup of 8 waves (heads of 64: of 4) holds 32 rows a wave of one kv head (row r = new token
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
// rarely rescaled. p is rounded to fp16 (relative 2^-11); its sum is not, since a
// block of small values has small p whatever its scores.
// LDS rows are swizzled by 16-byte pieces, so that lanes that read together hit
// different banks.
// Bound by the matrix cores and the exponentials beside them.
#include <type_traits>

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

constexpr float kSlack = 8.0f;       // how far (powers of two) the maximum may run ahead of the reference

// The swizzle of a key row and of a value row: 16-byte piece -> place. Keys of
// 128 elements fill a line of the 64 banks, the others half of one: any 16
// lanes that read together hit all of the line's 16 places.
template <int D>
__device__ __forceinline__ int key_place(int token, int piece) {
  return D == 128 ? piece ^ (token & 15) : piece ^ ((token >> 1) & 7);
}
__device__ __forceinline__ int value_place(int d, int piece) { return piece ^ ((d >> 1) & 7); }

// A barrier for what is exchanged through LDS: loads from memory stay in flight across it.
// Nothing is scheduled across it: a phase keeps to its own unit.
__device__ __forceinline__ void phase_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  __builtin_amdgcn_sched_barrier(0);
}

template <int D, int FMT>
__global__ __launch_bounds__(2 * attn_rows(D), 2) void k_attn_rows(AttnArgs A) {
  constexpr int kWaves = attn_rows(D) / 32;
  constexpr int THREADS = 64 * kWaves, KS = D / 16, DT = D / 32;
  constexpr int PIECES = kKvBlock * D / 16;               // 16-byte pieces of codes of a block's keys (and values)
  constexpr int LOADS = (2 * PIECES + THREADS - 1) / THREADS;
  static_assert(2 * PIECES % THREADS == 0 && PIECES % 64 == 0, "a wave loads keys or values, not both");
  __shared__ __attribute__((aligned(16))) _Float16 lk[2][kKvBlock * D], lv[2][kKvBlock * D];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 31, f = lane >> 5;

  // workgroup -> (row tile, the last first: it sees the most; sequence; split; kv head)
  int w = (int)blockIdx.x;
  const int h = w % A.kv.hk;
  w /= A.kv.hk;
  const int split = w % A.splits;
  w /= A.splits;
  const int s = w % A.b.seqs, rt = A.row_tiles - 1 - w / A.b.seqs;
  // The blocks' numbers come first: their codes are what the workgroup waits for. Loads are unconditional, here and
  // below, so that nothing waits for them before they are used: what does not exist or is not coded is read from a
  // place that does and not looked at.
  const int b0 = split * A.chunk, table_last = A.b.width - 1;
  const uint32_t blocks = (uint32_t)A.kv.blocks;
  const int32_t* table = A.b.table + (int64_t)s * A.b.width;
  const auto id_of = [&](int t) { return table[min(b0 + t, table_last)]; };
  const auto head_of = [&](int id) { return (int64_t)((uint32_t)id < blocks ? id : 0) * A.kv.hk + h; };
  int id_t = id_of(0), id_1 = id_of(1), id_2 = id_of(2), id_3 = id_of(3);   // blocks t .. t + 3
  const Seq sq = seq_of(A.b, A.kv, s);
  const int rows = sq.n * A.group, row0 = rt * 32 * kWaves;
  if (row0 >= rows) return;
  const int len = sq.cap;

  struct Codes {
    uint4 p[LOADS];
  };
  const auto keys = [&](int i) {   // whether the wave's i-th pieces are of the keys
    return PIECES % THREADS == 0 ? i * THREADS < PIECES : wave < kWaves / 2;
  };
  const auto load = [&](Codes& codes, int id_k, int id_v) {
    const uint8_t* kp = A.kv.kc + head_of(id_k) * (kKvBlock * D);
    const uint8_t* vp = A.kv.vc + head_of(id_v) * (kKvBlock * D);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      codes.p[i] = *reinterpret_cast<const uint4*>((keys(i) ? kp : vp) + (tid + i * THREADS) % PIECES * 16);
  };
  Codes codes, before;   // of the stage to lay next: the keys of block t + 2 and the values of block t + 1
  load(before, id_t, id_t);
  load(codes, id_1, id_t);
  float ks = A.kv.ks[head_of(id_t)], vs = A.kv.vs[head_of(id_t)];   // of block t, as loaded, a turn ahead

  // this lane's row
  const int r = row0 + 32 * wave + c;
  const int rr = r < rows ? r : row0;
  const int tok = rr / A.group, hh = rr % A.group;
  const int end = r >= rows ? 0 : A.causal ? max(len - sq.n + tok + 1, 0) : len;
  half8_t qf[KS];
  const _Float16* qp = A.q.p + (int64_t)(sq.q0 + tok) * A.q.stride + (int64_t)(h * A.group + hh) * D;
#pragma unroll
  for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const half8_t*>(qp + 16 * k + 8 * f);
  const float scale2 = fabsf(A.scale2);
  // tokens that the workgroup and this wave see, and those that every row of the wave sees: rows see more the later they are
  const auto end_of = [&](int row) { return A.causal ? max(len - sq.n + row / A.group + 1, 0) : len; };
  const int group_end = end_of(min(rows, row0 + 32 * kWaves) - 1);
  const int wave_row = row0 + 32 * wave;
  const int wave_end = wave_row < rows ? end_of(min(rows, wave_row + 32) - 1) : 0;
  const int wave_all = wave_row < rows ? end_of(wave_row) : 0;
  const int nblk = (group_end + kKvBlock - 1) / kKvBlock;
  const int b1 = min(nblk, b0 + A.chunk);
  const int open_blk = len / kKvBlock;

  float16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNoMax, l = 0.0f;

  const int n = max(b1 - b0, 0);
  // Lays stage t into LDS (keys of block t + 1, values of block t): coded blocks only (FAST), or whatever the blocks are.
  const auto lay = [&](auto fast_, const Codes& codes, int t) {
    constexpr bool FAST = decltype(fast_)::value;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int p = tid + i * THREADS;
      const bool is_k = keys(i);
      const int b = b0 + t + (is_k ? 1 : 0);
      if (!FAST && (b < b0 || b >= b1)) continue;
      _Float16* dst = is_k ? lk[(t + 1) & 1] : lv[t & 1];
      // this piece of 16 codes: two places of 8 elements in the row of a token or of a value element
      const int q = p % PIECES, per = is_k ? D / 16 : kKvBlock / 16, row = q / per, piece = 2 * (q % per);
      const int at0 = is_k ? row * D + 8 * key_place<D>(row, piece) : row * kKvBlock + 8 * value_place(row, piece);
      const int at1 = is_k ? row * D + 8 * key_place<D>(row, piece + 1) : row * kKvBlock + 8 * value_place(row, piece + 1);
      half8_t lo, hi;
      if (FAST || b != open_blk) {
        lo = widen8<FMT>(codes.p[i].x, codes.p[i].y);
        hi = widen8<FMT>(codes.p[i].z, codes.p[i].w);
      } else {   // the open block is fp16; tokens from `left` on are not the sequence's and may be no numbers
        const int left = len - b * kKvBlock;
        const half8_t* src = reinterpret_cast<const half8_t*>(
            (is_k ? A.kv.kt : A.kv.vt) + ((int64_t)max(sq.slot, 0) * A.kv.hk + h) * (kKvBlock * D) + 16 * q);
        lo = src[0];
        hi = src[1];
        if (!is_k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (8 * piece + e >= left) lo[e] = (_Float16)0.0f;
            if (8 * piece + 8 + e >= left) hi[e] = (_Float16)0.0f;
          }
        }
      }
      *reinterpret_cast<half8_t*>(dst + at0) = lo;
      *reinterpret_cast<half8_t*>(dst + at1) = hi;
    }
  };

  const int ktok = 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);
  int vat[4], kat[KS];   // where this lane's fragments lie: value pieces, key pieces
#pragma unroll
  for (int i = 0; i < 4; ++i) vat[i] = c * kKvBlock + 8 * value_place(c, 2 * i + f);
#pragma unroll
  for (int k = 0; k < KS; ++k) kat[k] = ktok * D + 8 * key_place<D>(ktok, 2 * k + f);

  struct Scores {
    float16_t t[2];   // t[x][8 y + j]: token 32 x + 16 y + 8 f + j of the block, this lane's row
  };
  Scores sa, sb;
  half8_t pf[2][2];
  const auto multiply_keys = [&](Scores& sc, const _Float16* src) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 16; ++i) sc.t[x][i] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        sc.t[x] = mfma32(*reinterpret_cast<const half8_t*>(src + kat[k] + 32 * D * x), qf[k], sc.t[x]);
  };
  const auto multiply_values = [&](const _Float16* src) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        o[d] = mfma32(*reinterpret_cast<const half8_t*>(src + vat[i] + 32 * kKvBlock * d), pf[i >> 1][i & 1], o[d]);
  };
  const auto largest = [&](const Scores& sc) {
    float top = sc.t[0][0];
#pragma unroll
    for (int i = 1; i < 32; ++i) top = fmaxf(top, sc.t[i >> 4][i & 15]);
    return max_halves(top);
  };
  const auto follow = [&](float top) {   // moves the reference where the maximum has run away from it
    if (__any(top > m + kSlack)) {
      const float now = fmaxf(m, top);
      const float shrink = __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= shrink;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= shrink;
    }
  };

  // Turn t: the weights of block t from its scores, the product with its values, and the scores of block t + 1; the
  // keys of block t + 2 and the values of block t + 1 are laid. X = t % 2.
  // The guarded turn, for a sequence's first and last blocks: whatever the rows see and whatever the blocks are.
  const auto turn_any = [&](int X, int t) {
    const int b = b0 + t;
    if (t < n && b * kKvBlock < wave_end) {
      float k1 = ks, v1 = vs;
      if (b == open_blk) k1 = v1 = 1.0f;
      if (!(b == open_blk ? sq.slot >= 0 : (uint32_t)id_t < blocks)) k1 = __builtin_nanf("");
      v1 = v1 == 0.0f ? kZeroScale : v1;
      const float mul = k1 * scale2, add = __builtin_amdgcn_logf(v1);
      const int left = end - b * kKvBlock - 8 * f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (16 * (i >> 3) + (i & 7) >= left) sa.t[i >> 4][i & 15] = -INFINITY;
      float top = largest(sa);
      const bool none = top == -INFINITY;
      top = none ? kNoMax : fmaf(top, mul, add);
      follow(top);
      const float off = add - m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float p = __builtin_amdgcn_exp2f(fmaf(sa.t[i >> 4][i & 15], mul, off));
        if (16 * (i >> 3) + (i & 7) >= left) p = 0.0f;   // again: a masked score times a NaN or zero scale is no weight
        sum += p;
        pf[i >> 4][(i >> 3) & 1][i & 7] = (_Float16)p;
      }
      l = fmaf(sum, __builtin_amdgcn_rcpf(v1), l);
      multiply_values(lv[X]);
    }
    if (t + 1 < n && (b + 1) * kKvBlock < wave_end) multiply_keys(sa, lk[X ^ 1]);
  };
  const auto next_blocks = [&](int t) {
    ks = A.kv.ks[head_of(id_1)];
    vs = A.kv.vs[head_of(id_1)];
    id_t = id_1;
    id_1 = id_2;
    id_2 = id_3;
    id_3 = id_of(t + 4);
  };
  // The order of a whole turn's instructions: fragments are read four ahead, and the exponentials and the rest of the
  // vector work go between the multiplications, which the two waves of a SIMD then keep fed.
  const auto interleave = [&]() {
    __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);   // LDS reads
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a multiplication
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);   // vector instructions
    }
#pragma unroll
    for (int i = 0; i < 4 * DT; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
    }
  };
  // The turn of blocks that every row of the wave sees whole, with coded blocks to lay: no branch but the reference's.
  float top = 0.0f;   // largest score of block t, before its scale
  const auto turn_whole = [&](Scores& now, Scores& next, int X, int t) {
    const float k1 = (uint32_t)id_t < blocks ? ks : __builtin_nanf(""), v1 = vs == 0.0f ? kZeroScale : vs;
    const float mul = k1 * scale2, add = __builtin_amdgcn_logf(v1);
    follow(fmaf(top, mul, add));
    const float off = add - m;
    next_blocks(t);
    multiply_keys(next, lk[X ^ 1]);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float p = __builtin_amdgcn_exp2f(fmaf(now.t[i >> 4][i & 15], mul, off));
      sum[i & 3] += p;
      pf[i >> 4][(i >> 3) & 1][i & 7] = (_Float16)p;
    }
    l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), __builtin_amdgcn_rcpf(v1), l);
    multiply_values(lv[X]);
    lay(std::true_type{}, codes, t + 1);
    load(codes, id_2, id_1);
    top = largest(next);
    if (D == 128) interleave();   // heads of 64 are 4 % faster in the compiler's own order, heads of 128 14 % slower
    phase_barrier();
  };
  if (n > 0) {   // a part of the cache that none of the rows sees is left out
    lay(std::false_type{}, before, -1);
    lay(std::false_type{}, codes, 0);
    load(codes, id_2, id_1);
    if (A.scale2 < 0.0f) {   // a negative scale turns the queries: scores can then be compared before they are scaled
#pragma unroll
      for (int k = 0; k < KS; ++k) qf[k] = -qf[k];
    }
    phase_barrier();
    if (b0 * kKvBlock < wave_end) multiply_keys(sa, lk[0]);
    // whole turns: block t seen whole, and no open block among those that are laid (what lies past the last block is laid
    // too, and not looked at)
    const int whole = min(min(wave_all / kKvBlock - b0, n), open_blk < b1 ? open_blk - b0 - 2 : n);
    int t = 0;
    if (whole > 1) top = largest(sa);
    phase_barrier();   // all have read the keys of block 0: the first turn lays those of block 2 in their place
    for (; t + 1 < whole; t += 2) {
      turn_whole(sa, sb, 0, t);
      turn_whole(sb, sa, 1, t + 1);
    }
    for (; t < n; ++t) {
      turn_any(t & 1, t);
      next_blocks(t);
      lay(std::false_type{}, codes, t + 1);
      load(codes, id_2, id_1);
      phase_barrier();
    }
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

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& A, int dim, int format, const AttnPlan& p, hipStream_t s) {
  const dim3 g((unsigned)p.groups), t(2 * attn_rows(dim));
  if (dim == 64) {
    if (format == MQ_KV_INT8) k_attn_rows<64, MQ_KV_INT8><<<g, t, 0, s>>>(A);
    else k_attn_rows<64, MQ_KV_E4M3><<<g, t, 0, s>>>(A);
  } else {
    if (format == MQ_KV_INT8) k_attn_rows<128, MQ_KV_INT8><<<g, t, 0, s>>>(A);
    else k_attn_rows<128, MQ_KV_E4M3><<<g, t, 0, s>>>(A);
  }
  return hipGetLastError();
}

}  // namespace mq
