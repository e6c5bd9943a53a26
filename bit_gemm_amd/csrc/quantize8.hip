// Rows and weights in 8 bits (include/mosaicq_head.h, mq_quantize8 and
// mq_pack8): e4m3 codes with a power-of-two scale for each block of 128.
//
// 16 lanes hold a block, 8 elements each: one 16-byte load a lane, the block's
// largest magnitude by four lane exchanges, one 8-byte store. Every value is
// read and written once; bound by HBM for many rows (4096 of 14336, 177 MB, 30 us,
// 5.9 TB/s; 2048 of 8192, 50 MB, 10.6 us, 4.8), by one load's way for few (16 of
// 4096 3.1 us); between them by both: 512 of 14336 (22 MB) 6.4 us.
#include "block_common.h"
#include "head_internal.h"
#include "q8.h"

namespace mq {
namespace {

// The workgroups of a launch (a launch takes fewer than 2^32 threads); each goes on in steps of the grid.
constexpr int64_t kMostGroups = 1 << 20;

// Eight elements from d on of a row of K, zero past its end.
__device__ __forceinline__ void take_row8(const _Float16* row, int64_t d, int64_t K, float* v) {
  if (d + 8 <= K) {
    const half8_t h = load8(row + d);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = d + i < K ? (float)row[d + i] : 0.0f;
  }
}

__device__ __forceinline__ uint32_t top8(const float* v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, q8_magnitude(v[i]));
  return q8_top16(top);
}

// A workgroup takes 16 blocks of a row.
__global__ __launch_bounds__(256) void k_quantize8(const _Float16* x, int64_t K, int64_t xs, uint8_t* codes, int64_t cs,
                                                   uint8_t* scales, int64_t ss, int Kt, int per_row, int64_t groups) {
  for (int64_t b = blockIdx.x; b < groups; b += gridDim.x) {
    const int64_t row = b / per_row;
    const int kt = 16 * (int)(b - row * per_row) + (int)(threadIdx.x >> 4), part = threadIdx.x & 15;
    const int64_t d = (int64_t)kQ8Block * kt + 8 * part;
    float v[8];
    take_row8(x + row * xs, d, K, v);
    const uint32_t byte = q8_scale(top8(v));
    if (kt < Kt) {
      *reinterpret_cast<uint2*>(codes + row * cs + d) = q8_codes(v, byte);
      if (part == 0) scales[row * ss + kt] = (uint8_t)byte;
    }
  }
}

// A workgroup makes a tile: 16 rows, 128 columns.
__global__ __launch_bounds__(256) void k_pack8(const _Float16* w, int64_t ws, W8 out, uint8_t* codes, uint8_t* scales) {
  const int64_t tiles = (int64_t)out.Nb * out.Kt;
  const int r = threadIdx.x >> 4, part = threadIdx.x & 15;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t rb = t / out.Kt, row = 16 * rb + r;
    const int kt = (int)(t - rb * out.Kt);
    float v[8] = {};
    if (row < out.N) take_row8(w + row * ws, (int64_t)kQ8Block * kt + 8 * part, out.K, v);
    const uint32_t byte = q8_scale(top8(v));
    // columns 8 part .. + 7: half part / 8 of the tile, lanes 16 ((part % 8) / 2) + r, the first or last 8 of their 16 bytes
    uint8_t* to = codes + 2048 * t + 1024 * (part >> 3) + 16 * (16 * ((part & 7) >> 1) + r) + 8 * (part & 1);
    *reinterpret_cast<uint2*>(to) = q8_codes(v, byte);
    if (part == 0) {
      uint8_t* sc = scales + 64 * (rb * out.Kq) + 4 * r;
      sc[64 * (int64_t)(kt >> 2) + (kt & 3)] = (uint8_t)byte;
      if (kt == out.Kt - 1)
        for (int k = out.Kt; k < 4 * out.Kq; ++k) sc[64 * (int64_t)(k >> 2) + (k & 3)] = 127;
    }
  }
}

}  // namespace

hipError_t launch_quantize8(const _Float16* x, int64_t M, int64_t K, int64_t xs, uint8_t* codes, int64_t cs,
                            uint8_t* scales, int64_t ss, hipStream_t s) {
  const int Kt = (int)((K + kQ8Block - 1) / kQ8Block), per_row = (Kt + 15) / 16;
  const int64_t groups = M * per_row;
  if (groups == 0) return hipSuccess;
  const unsigned grid = (unsigned)(groups < kMostGroups ? groups : kMostGroups);
  k_quantize8<<<dim3(grid), dim3(256), 0, s>>>(x, K, xs, codes, cs, scales, ss, Kt, per_row, groups);
  return hipGetLastError();
}

hipError_t launch_pack8(const _Float16* w, int64_t ws, const W8& out, hipStream_t s) {
  const int64_t tiles = (int64_t)out.Nb * out.Kt;
  const unsigned grid = (unsigned)(tiles < kMostGroups ? tiles : kMostGroups);
  k_pack8<<<dim3(grid), dim3(256), 0, s>>>(w, ws, out, const_cast<uint8_t*>(out.codes), const_cast<uint8_t*>(out.scales));
  return hipGetLastError();
}

}  // namespace mq
