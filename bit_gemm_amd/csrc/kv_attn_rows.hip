// Attention over the 8-bit key/value cache for many query rows: prompts and
// their pieces (kv_attn.hip holds the kernel for few rows and the join).
//
// A workgroup of 8 waves (heads of 64: of 4) holds 32 rows a wave of one kv
// head (row r = new token r / g, query head r % g, so the g heads that share the
// keys share the tile) and walks the 64-token blocks they see. A block's codes are loaded
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
// reference m is laid 11 below the running maximum and follows it only when that
// has grown by more than 2^4 (p then reaches 2^15 at most, inside fp16), so the
// sums are rarely rescaled. p is rounded to fp16 (relative 2^-11, down to 2^-25 of
// the largest); its sum is not, since a block of small values has small p whatever
// its scores.
// LDS rows are swizzled by 16-byte pieces, so that lanes that read together hit
// different banks.
// Bound by the matrix cores and the exponentials beside them: a block of a
// workgroup takes 1.88 us with heads of 128 (all the GPU: 1.1 PFLOP/s, what a large
// product of matrices reaches) and 1.3 us with heads of 64 (0.8; the exponentials
// are as many for half the products). With their starts, ends and the blocks on the
// diagonal: a prompt of 4096, 32 query and 8 kv heads of 128 (137 GFLOP): 142 us.
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

// How far (powers of two) the maximum may grow before the reference follows. More leaves fewer bits below the largest
// weight, less rescales more often: 2, 4 and 8 took 143.8, 141.9 and 141.9 us for a prompt of 4096, 96.7, 94.9 and 93.9 us
// for 8 prompts of 500 to 1000 (32 query and 8 kv heads of 128).
constexpr float kSlack = 4.0f;

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

// The kernel's arguments, read anew.
__device__ __forceinline__ AttnArgs arguments() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)p;
}

// What a workgroup does for one row tile of a kv head: blocks from .. to - 1 of those that its rows see, written out where
// that is all, else into the workspace, unnormalised, each row where place_of(its number in q, in the tile) says. AGAIN:
// the arguments are read anew for that, so that the tile's loop has the scalar registers to itself (in the kernel of
// slices, that is: its turns are 8 % faster so).
template <int D, int FMT, bool AGAIN, typename PlaceOf>
__device__ __forceinline__ void attend(const AttnArgs& A, _Float16 (&lk)[2][kKvBlock * D], _Float16 (&lv)[2][kKvBlock * D],
                                       int tid, int s, int rt, int h, int from, int to, bool all, PlaceOf place_of) {
  constexpr int kWaves = attn_rows(D) / 32;
  constexpr int THREADS = 64 * kWaves, KS = D / 16, DT = D / 32;
  constexpr int PIECES = kKvBlock * D / 16;               // 16-byte pieces of codes of a block's keys (and values)
  constexpr int LOADS = (2 * PIECES + THREADS - 1) / THREADS;
  static_assert(2 * PIECES % THREADS == 0 && PIECES % 64 == 0, "a wave loads keys or values, not both");
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 31, f = lane >> 5;

  // The blocks' numbers come first: their codes are what the workgroup waits for. Loads are unconditional, here and
  // below, so that nothing waits for them before they are used: what does not exist or is not coded is read from a
  // place that does and not looked at.
  const int b0 = from, table_last = A.b.width - 1;
  const uint32_t blocks = (uint32_t)A.kv.blocks;
  const int32_t* table = A.b.table + (int64_t)s * A.b.width;
  const auto id_of = [&](int t) { return unwritten(table + min(b0 + t, table_last)); };
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
  float ks = unwritten(A.kv.ks + head_of(id_t)), vs = unwritten(A.kv.vs + head_of(id_t));   // of block t, as loaded, a turn ahead

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
  const int b1 = min(nblk, to);
  const int open_blk = len / kKvBlock;

  float16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.0f;
  float m = kNoMax, l = 0.0f;

  const int n = max(b1 - b0, 0);
  // Lays stage t into LDS (keys of block t + 1, values of block t): coded blocks only (FAST), or whatever the blocks are.
  const auto lay = [&](auto fast_, const Codes& codes, int t, int odd) {   // odd: t % 2, known where the code is laid out
    constexpr bool FAST = decltype(fast_)::value;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int p = tid + i * THREADS;
      const bool is_k = keys(i);
      const int b = b0 + t + (is_k ? 1 : 0);
      if (!FAST && (b < b0 || b >= b1)) continue;
      _Float16* dst = is_k ? lk[odd ^ 1] : lv[odd];
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
    if (__any(top > m + kMaxWeight)) {
      const float now = fmaxf(m, reference(top, kMaxWeight - kSlack));
      const float shrink = __builtin_amdgcn_exp2f(m - now);
      m = now;
      l *= shrink;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= shrink;
    }
  };
  // A weight is 2^(s mul + off) with off = add - m, one operation a score. Its rounding is that of m, which is nothing for
  // scores of usual size; where they are so large that a step of fp32 is whole powers of two, the difference of the score
  // and m is taken first.
  const auto far_scores = [&](Scores& sc, float top, float add, float& mul, float& off) {
    if (__any(fabsf(top) > kFar)) {
#pragma unroll
      for (int i = 0; i < 32; ++i) sc.t[i >> 4][i & 15] = fmaf(sc.t[i >> 4][i & 15], mul, add) - m;
      mul = 1.0f;
      off = 0.0f;
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
      float mul = k1 * scale2;
      const float add = __builtin_amdgcn_logf(v1);
      const int left = end - b * kKvBlock - 8 * f;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (16 * (i >> 3) + (i & 7) >= left) sa.t[i >> 4][i & 15] = -INFINITY;
      float top = largest(sa);
      const bool none = top == -INFINITY;
      top = none ? kNoMax : fmaf(top, mul, add);
      follow(top);
      float off = add - m;
      far_scores(sa, top, add, mul, off);
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
    ks = unwritten(A.kv.ks + head_of(id_1));
    vs = unwritten(A.kv.vs + head_of(id_1));
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
    float mul = k1 * scale2;
    const float add = __builtin_amdgcn_logf(v1), peak = fmaf(top, mul, add);
    follow(peak);
    float off = add - m;
    far_scores(now, peak, add, mul, off);
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
    lay(std::true_type{}, codes, t + 1, X ^ 1);
    load(codes, id_2, id_1);
    top = largest(next);
    if (D == 128) interleave();   // heads of 64 are 4 % faster in the compiler's own order, heads of 128 14 % slower
    phase_barrier();
  };
  if (n > 0) {   // a part of the cache that none of the rows sees is left out
    lay(std::false_type{}, before, -1, 1);
    lay(std::false_type{}, codes, 0, 0);
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
      lay(std::false_type{}, codes, t + 1, (t + 1) & 1);
      load(codes, id_2, id_1);
      phase_barrier();
    }
  }

  if (end > 0) l += zero_if_finite(qf);
  l = sum_halves(l);
  if (r >= rows) return;
  const AttnArgs Z = AGAIN ? arguments() : A;
  const int64_t at_tok = (AGAIN ? seq_of(Z.b, Z.kv, s).q0 : sq.q0) + tok;
  if (all) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    _Float16* out = Z.out.p + at_tok * Z.out.stride + (int64_t)(h * Z.group + hh) * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4_t v = {o[d][i] * inv, o[d][i + 1] * inv, o[d][i + 2] * inv, o[d][i + 3] * inv};
        store4(reinterpret_cast<uint16_t*>(out + 32 * d + 2 * i + 4 * f), v, 4, true);
      }
  } else {
    const int64_t row = place_of(at_tok * Z.hq + h * Z.group + hh, 32 * wave + c);
    float* out = Z.ws_o + row * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4_t*>(out + 32 * d + 2 * i + 4 * f) =
            (float4_t){o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (f == 0) Z.ws_ml[row] = make_float2(m, l);
  }
}

// One row tile a workgroup, or one split of its blocks; the last rows first: they see the most.
template <int D, int FMT>
__global__ __launch_bounds__(2 * attn_rows(D), 2) void k_attn_rows(AttnArgs A) {
  __shared__ __attribute__((aligned(16))) _Float16 lk[2][kKvBlock * D], lv[2][kKvBlock * D];
  int w = (int)blockIdx.x;
  const int h = w % A.kv.hk;
  w /= A.kv.hk;
  const int split = w % A.splits;
  w /= A.splits;
  attend<D, FMT, false>(A, lk, lv, threadIdx.x, w % A.b.seqs, A.row_tiles - 1 - w / A.b.seqs, h, split * A.chunk,
                        (split + 1) * A.chunk, A.splits == 1, [&](int64_t row, int) { return row * A.splits + split; });
}

// Slices. Where there are few row tiles for the GPU their work is laid end to end -- sequence by sequence, kv head by kv
// head, tile by tile -- and cut into slices of the same size, one a workgroup, whatever tiles the cuts fall into: lengths
// differ, and whole tiles, or parts of one size, leave most of the GPU waiting for the last ones (9 sequences of 3000 to
// 12000 tokens with 200 to 700 new ones, heads of 64: 170 us, in two splits a tile 270). The host does not know
// the lengths, so every workgroup finds its own slice on the line. A tile costs the blocks that it sees, as a linear
// function of its number in a head whose sums have a closed form, and kExtra for its start and end. Costs are fp32: what
// matters is that the same cut comes out the same in both workgroups that make it, so nothing here is fused or
// reordered, and that places follow each other as their costs do, which rounding keeps.
constexpr float kExtra = 4.0f, kLeast = 8.0f;   // blocks; a slice is at least kLeast long (8, and 5 or 12: within 2 %)
constexpr int kEdge = 2;                        // a cut this near to an end of a tile is made there

struct Work {
  float base, slope, head;   // cost of a tile: base + slope (its number + 1); cost of all tiles of a kv head
  int tiles;
};
__device__ __forceinline__ float cost_of_first(const Work& w, int tiles) {
#pragma clang fp contract(off)
  const float t = (float)tiles;
  return t * w.base + t * (t + 1.0f) * (0.5f * w.slope);
}
template <int TR>
__device__ __forceinline__ Work work_of(const AttnArgs& A, int n, int cap) {
#pragma clang fp contract(off)
  Work w;
  w.tiles = min(A.row_tiles, (int)(((int64_t)n * A.group + TR - 1) / TR));
  w.base = (float)(A.causal ? max(cap - n, 0) : cap) * (1.0f / kKvBlock) + kExtra;
  w.slope = A.causal ? (float)TR / (float)(kKvBlock * A.group) : 0.0f;
  w.head = cost_of_first(w, w.tiles);
  return w;
}
// Blocks of a tile, at least one: a tile that sees nothing is still written.
template <int TR>
__device__ __forceinline__ int blocks_of(const AttnArgs& A, int n, int cap, int rt) {
  const int last = (int)min((int64_t)n * A.group, (int64_t)(rt + 1) * TR) - 1;
  const int end = A.causal ? max(cap - n + last / A.group + 1, 0) : cap;
  return max((end - 1) / kKvBlock + 1, 1);
}

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// A place on the line: block `block` of row tile rt of kv head h of sequence s; s = seqs: its end.
struct Place {
  int s, h, rt, block;
};

__device__ __forceinline__ Place uniform(const Place& p) {
  return {__builtin_amdgcn_readfirstlane(p.s), __builtin_amdgcn_readfirstlane(p.h), __builtin_amdgcn_readfirstlane(p.rt),
          __builtin_amdgcn_readfirstlane(p.block)};
}
// The tile after p's, in a head of `tiles`.
__device__ __forceinline__ Place after(const AttnArgs& A, const Place& p, int tiles) {
  if (p.rt + 1 < tiles) return {p.s, p.h, p.rt + 1, 0};
  if (p.h + 1 < A.kv.hk) return {p.s, p.h + 1, 0, 0};
  int s = p.s + 1;
  while (s < A.b.seqs && seq_of(A.b, A.kv, s).n == 0) ++s;
  return {s, 0, 0, 0};
}

template <int TR>
struct Line {
  const AttnArgs& A;
  struct Lanes {         // 64 sequences, one a lane
    int n, cap;          // new tokens, all tokens
    float cost, before, up_to;   // of the sequence; of those of the 64 before it; of these and it
  } front;               // the first 64
  float total;

  __device__ __forceinline__ Lanes scan(int s0) const {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63, s = s0 + lane;
    Lanes l = {0, 0, 0.0f, 0.0f, 0.0f};
    if (s < A.b.seqs) {
      const Seq q = seq_of(A.b, A.kv, s);
      l.n = q.n;
      l.cap = q.cap;
      l.cost = work_of<TR>(A, q.n, q.cap).head * (float)A.kv.hk;
    }
    l.up_to = l.cost;
    for (int d = 1; d < min(A.b.seqs - s0, 64); d <<= 1) {
      const float v = __shfl_up(l.up_to, d);
      if (lane >= d) l.up_to += v;
    }
    const float v = __shfl_up(l.up_to, 1);
    l.before = lane > 0 ? v : 0.0f;
    return l;
  }
  __device__ __forceinline__ float sum(const Lanes& l, int s0) const { return lane_of(l.up_to, min(A.b.seqs - s0, 64) - 1); }
  __device__ __forceinline__ explicit Line(const AttnArgs& a) : A(a) {
    front = scan(0);
    total = sum(front, 0);
    for (int s0 = 64; s0 < A.b.seqs; s0 += 64) total += sum(scan(s0), s0);
  }
  // The place where a cost of x has been laid.
  __device__ __forceinline__ Place at(float x) const {
#pragma clang fp contract(off)
    Lanes l = front;
    int s0 = 0;
    uint64_t here;
    while (!(here = __ballot(x < l.up_to && l.cost > 0.0f))) {
      x -= sum(l, s0);
      s0 += 64;
      if (s0 >= A.b.seqs) return {A.b.seqs, 0, 0, 0};
      l = scan(s0);
    }
    const int lane = (int)__builtin_ctzll(here);
    x -= lane_of(l.before, lane);
    const int n = __builtin_amdgcn_readlane(l.n, lane), cap = __builtin_amdgcn_readlane(l.cap, lane);
    const Work w = work_of<TR>(A, n, cap);
    x = fmaxf(x, 0.0f);
    const int h = min((int)(x * __builtin_amdgcn_rcpf(w.head)), A.kv.hk - 1);
    x -= (float)h * w.head;
    int rt = 0, above = w.tiles;   // the last tile that begins at x or before
    while (above - rt > 1) {
      const int mid = (rt + above) >> 1;
      if (cost_of_first(w, mid) <= x) rt = mid;
      else above = mid;
    }
    const float begin = cost_of_first(w, rt), tile = cost_of_first(w, rt + 1) - begin;
    const int nb = blocks_of<TR>(A, n, cap, rt);
    const float part = fminf(fmaxf((x - begin) * __builtin_amdgcn_rcpf(tile), 0.0f), 1.0f);
    const int block = (int)(part * (float)nb);
    const Place p = {s0 + lane, __builtin_amdgcn_readfirstlane(h), __builtin_amdgcn_readfirstlane(rt),
                     __builtin_amdgcn_readfirstlane(block < kEdge ? 0 : block)};
    return p.block > 0 && nb - block < kEdge ? after(A, p, w.tiles) : p;
  }
};

// Slices are laid on every XCD in turn: slice w is workgroup (w % per) * 8 + w / per, so that the slices of an XCD are
// neighbours and share what they read.
__device__ __forceinline__ int group_of(int w, int per) { return w % per * 8 + w / per; }

template <int D, int FMT>
__global__ __launch_bounds__(2 * attn_rows(D), 2) void k_attn_slices(AttnArgs A) {
  constexpr int TR = attn_rows(D);
  __shared__ __attribute__((aligned(16))) _Float16 lk[2][kKvBlock * D], lv[2][kKvBlock * D];
  // What is to be known after a tile waits in LDS: the tile's loop has no register to spare for it.
  __shared__ struct {
    Place at, end;
    SlicePart mark;
  } next;
  {
    const Line<TR> line(A);
    const int slices = (int)fminf(fmaxf(line.total * (1.0f / kLeast), 1.0f), (float)gridDim.x);
    const int per = (slices + 7) / 8, w = (int)blockIdx.x % 8 * per + (int)blockIdx.x / 8;
    const bool mine = (int)blockIdx.x / 8 < per && w < slices;
    Place at = {A.b.seqs, 0, 0, 0}, end = at;
    const float each = line.total / (float)slices;
#pragma unroll 1
    for (int k = 0; mine && k < 2; ++k) {
      at = end;
      end = w + k < slices ? line.at(each * (float)(w + k)) : Place{A.b.seqs, 0, 0, 0};
    }
    if (threadIdx.x == 0) {
      next.at = at;
      next.end = end;
      next.mark = {0, 0, 0, 0, w, slices};
    }
  }
  while (true) {
    __syncthreads();
    const Place at = uniform(next.at), end = uniform(next.end);
    if (at.s >= A.b.seqs) break;
    const Seq q = seq_of(A.b, A.kv, at.s);
    const bool last = at.s == end.s && at.h == end.h && at.rt == end.rt;
    const int nb = blocks_of<TR>(A, q.n, q.cap, at.rt), to = last ? end.block : nb;
    if (to == 0) break;   // a cut between two tiles
    __syncthreads();
    if (threadIdx.x == 0) {
      if (at.block > 0) next.mark.flags |= to == nb ? kPartOf | kPartEnds : kPartOf;
      if (at.block == 0 && to < nb) {
        next.mark.flags |= kPartBegins;
        next.mark.s = at.s;
        next.mark.h = at.h;
        next.mark.rt = at.rt;
      }
      next.at = last ? Place{A.b.seqs, 0, 0, 0} : after(A, at, work_of<TR>(A, q.n, q.cap).tiles);
    }
    // nothing that a tile makes from these is kept for the next one: registers are scarce
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int slot = 2 * (int)blockIdx.x + (at.block == 0);
    attend<D, FMT, true>(arguments(), lk, lv, tid, at.s, at.rt, at.h, at.block, to, at.block == 0 && to == nb,
                         [&](int64_t, int r) { return (int64_t)slot * TR + r; });
  }
  if (threadIdx.x == 0) A.ws_parts[blockIdx.x] = next.mark;
}

// Joins the parts of the tile that begins in a workgroup's slice and does not end there: the workgroup's own, then those
// of the slices that follow, up to the one that ends the tile, added in that order.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join_slices(AttnArgs A) {
  constexpr int TR = attn_rows(D), X = D / 4, R = 256 / X;   // threads of a row; rows of a workgroup
  const int i = (int)blockIdx.x;
  const SlicePart mark = A.ws_parts[i];
  if (!(mark.flags & kPartBegins)) return;
  // how many parts: all lanes look, also those without a row
  const int per = (mark.slices + 7) / 8, lane = threadIdx.x & 63;
  int parts = 1;
  for (int w = mark.w + 1; w < mark.slices; w += 64) {
    const bool ends = w + lane >= mark.slices || (A.ws_parts[group_of(w + lane, per)].flags & kPartEnds);
    const uint64_t any = __ballot(ends);
    parts += any ? (int)__builtin_ctzll(any) + 1 : 64;
    if (any) break;
  }
  parts = min(parts, mark.slices - mark.w);
  const Seq q = seq_of(A.b, A.kv, mark.s);
  const int x = threadIdx.x % X, r = (int)blockIdx.y * R + threadIdx.x / X;
  const int64_t row = (int64_t)mark.rt * TR + r;
  if (row >= (int64_t)q.n * A.group) return;
  float top = kNoMax, total = 0.0f;
  float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p = 0; p < parts; p += 4) {   // four at a time
    float2 ml[4];
    float4_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int g = group_of(mark.w + min(p + j, parts - 1), per);
      const int64_t place = (int64_t)(2 * g + (p + j == 0)) * TR + r;
      ml[j] = A.ws_ml[place];
      o[j] = reinterpret_cast<const float4_t*>(A.ws_o)[place * X + x];
    }
    float now = top;
#pragma unroll
    for (int j = 0; j < 4; ++j) now = fmaxf(now, p + j < parts ? ml[j].x : kNoMax);
    const float shrink = __builtin_amdgcn_exp2f(top - now);
    top = now;
    total *= shrink;
    acc *= shrink;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p + j >= parts) continue;
      const float f = __builtin_amdgcn_exp2f(ml[j].x - top);
      total += ml[j].y * f;
      acc += o[j] * f;
    }
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t tok = q.q0 + row / A.group, hh = mark.h * A.group + row % A.group;
  store4(reinterpret_cast<uint16_t*>(A.out.p + tok * A.out.stride + hh * D + 4 * x), acc * inv, 4, true);
}

template <int D, int FMT>
hipError_t go(const AttnArgs& A, const AttnPlan& p, hipStream_t s) {
  const dim3 g((unsigned)p.groups), t(2 * attn_rows(D));
  if (!p.slices) {
    k_attn_rows<D, FMT><<<g, t, 0, s>>>(A);
    return hipGetLastError();
  }
  k_attn_slices<D, FMT><<<g, t, 0, s>>>(A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_attn_join_slices<D><<<dim3((unsigned)p.groups, attn_rows(D) * D / 1024), dim3(256), 0, s>>>(A);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs& A, int dim, int format, const AttnPlan& p, hipStream_t s) {
  if (dim == 64) return format == MQ_KV_INT8 ? go<64, MQ_KV_INT8>(A, p, s) : go<64, MQ_KV_E4M3>(A, p, s);
  return format == MQ_KV_INT8 ? go<128, MQ_KV_INT8>(A, p, s) : go<128, MQ_KV_E4M3>(A, p, s);
}

}  // namespace mq
