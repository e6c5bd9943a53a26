// Internal declarations of the head's operators (include/mosaicq_head.h):
// what the host hands to the kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/mosaicq_head.h"
#include "head_plan.h"

namespace mq {

// 8-bit rows, as mq_quantize8 writes them.
struct Rows8 {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t stride, sstride;   // bytes between rows
};

// 8-bit weights in the order of mq_w8.
struct W8 {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t N, K;
  int Nb, Kt, Kq;            // blocks of 16 rows, blocks of 128 columns, fours of those
};

hipError_t launch_quantize8(const _Float16* x, int64_t M, int64_t K, int64_t xs, uint8_t* codes, int64_t cs,
                            uint8_t* scales, int64_t ss, hipStream_t s);
hipError_t launch_pack8(const _Float16* w, int64_t ws, const W8& out, hipStream_t s);

hipError_t launch_linear8(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, void* ws,
                          const Linear8Plan& plan, hipStream_t s);

size_t sample_workspace(int64_t rows, int64_t vocab, int fp32);
hipError_t launch_sample(const mq_sample_args& a, void* ws, hipStream_t s);

}  // namespace mq
