// What the attention kernels share: codes to fp16, their arguments.
#pragma once
#include "block_common.h"

namespace mq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -3.4028235e38f;   // the reference before the first visible token: finite, and no score is below
constexpr float kMaxWeight = 15.0f;  // weights 2^(t - m) reach 2^15 at most, inside fp16
constexpr float kFar = 1 << 20;      // up to here a few powers of two can be taken from a score with little rounding
constexpr float kZeroScale = 1.0f / (1 << 30);   // stands for the scale of values that are all zero

// The reference for weights whose largest score is top: `by` below it, so that the largest weight is 2^by and one of
// 2^-(14 + by) of it is still a normal fp16 number. Thousands of weights that small may be the whole output, where the
// largest belong to values of about zero (by = 0: weights of 2^-24.5 of the largest were off by 41 %, smaller ones lost).
__device__ __forceinline__ float reference(float top, float by) { return fabsf(top) < kFar ? top - by : top; }

// 8 codes (two dwords) as fp16, exactly.
template <int FMT>
__device__ __forceinline__ half8_t widen8(uint32_t a, uint32_t b) {
  u32x4_t r;
  if (FMT == MQ_KV_E4M3) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
  } else {
    // code + 128 as the low byte of fp16 1024 + u, then - 1152
    const half2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    const uint32_t ua = a ^ 0x80808080u, ub = b ^ 0x80808080u, m = 0x64646464u;
    r.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m, ua, 0x04010400u)) - bias);
    r.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m, ua, 0x04030402u)) - bias);
    r.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m, ub, 0x04010400u)) - bias);
    r.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m, ub, 0x04030402u)) - bias);
  }
  return __builtin_bit_cast(half8_t, r);
}

// 0, or NaN where one of a lane's N pieces of a query is not finite. A row's sum of weights takes it in at the end: such
// a query has no finite score, and where all are -Inf nothing else would tell it from a row that sees nothing.
template <int N>
__device__ __forceinline__ float zero_if_finite(const half8_t (&q)[N]) {
  half8_t z = q[0] * (_Float16)0.0f;
#pragma unroll
  for (int i = 1; i < N; ++i) z += q[i] * (_Float16)0.0f;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += (float)z[i];
  return sum;
}

// What a workgroup of k_attn_slices says of its slice, for the join: flags, the tile that begins in it and goes on, the
// slice's number and how many there are.
enum { kPartOf = 1, kPartEnds = 2, kPartBegins = 4 };   // it goes on with a tile; that tile ends in it; one begins and goes on
struct SlicePart {
  int flags, s, h, rt, w, slices;
};

struct AttnArgs {
  KvView kv;
  BatchView b;
  RowsIn q;
  RowsOut out;
  int hq, group, causal;
  float scale2;     // scale log2(e): scores are in units of the 2-based exponent
  int row_tiles, chunk, splits;
  float* ws_o;      // unnormalised sums, [tokens][q heads][splits][D]; of slices [workgroups][2][rows][D]
  float2* ws_ml;    // likewise (m, l); l = 0: nothing seen
  SlicePart* ws_parts;   // [workgroups]
};

// The kernel for many query rows (kv_attn_rows.hip).
hipError_t launch_attn_rows(const AttnArgs& A, int dim, int format, const AttnPlan& p, hipStream_t s);

}  // namespace mq
