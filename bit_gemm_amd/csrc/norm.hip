// Norms before and after a block with its gate and residual
// (include/mosaicq_block.h, mq_norm_residual and mq_norm_residual_q8).
//
//   r' = alpha r + beta g (y / rms(y)) (w_post + o),  h = (r' / rms(r')) (w_pre + o)
//
// One workgroup a row, the row in registers from the first read to the last
// write, so every input is read once; two sums over the row, of y^2 and of
// r'^2, in fp32, a thread's own elements first, then the lanes of a wave, then
// the waves in order. Bound by HBM for many rows (y, r, gate read, r', h
// written); by the two dependent sums and the load before them for few. 4096
// rows of 8192, fp32 residual and a gate (470 MB): 87 us, 5.4 TB/s, the rate of
// a large copy; 16 rows of 4096: 4.3 us. Rows past 32768 elements spill. With
// h in 8 bits (436 MB) 88 us, 4.9 TB/s, and 4.0 us: each code is taken from its
// block's 16 lanes, where a quantizer after the norm would read h again (4096
// rows of 8192 in fp16: 102 MB more).
#include "block_common.h"
#include "q8.h"

namespace mq {
namespace {

// Where 8-bit rows get their scales; h_out and h_stride are the codes' then.
struct ScalesOut {
  uint8_t* p;
  int64_t stride;
};

template <int WAVES>
__device__ __forceinline__ float sum_group(float v, float* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += lds[w];
  return t;
}

// 8 elements from p, or the first `left` of them one by one where the row ends; rows may start anywhere.
__device__ __forceinline__ void take8(const _Float16* p, int left, float* v) {
  if (left >= 8) {
    const half8_t h = load8(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)p[i] : 0.0f;
  }
}
__device__ __forceinline__ void take8(const float* p, int left, float* v) {
  if (left >= 8) {
    const float4_t a = reinterpret_cast<const float4_any_t*>(p)[0], b = reinterpret_cast<const float4_any_t*>(p + 4)[0];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[i + 4] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void put8(_Float16* p, int left, const float* v) {
  if (left >= 8) {
    half8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    store8(p, h);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (_Float16)v[i];
  }
}
__device__ __forceinline__ void put8(float* p, int left, const float* v) {
  if (left >= 8) {
    reinterpret_cast<float4_any_t*>(p)[0] = (float4_t){v[0], v[1], v[2], v[3]};
    reinterpret_cast<float4_any_t*>(p + 4)[0] = (float4_t){v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}

// CH pieces of 8 elements a thread. Multiply-adds are written out, so that all
// instances give the same bits. Q8: h goes out as 8-bit rows, coded from its
// fp32 values (one rounding); a block of 128 lies in 16 lanes that follow each
// other, so its largest magnitude takes four lane exchanges and no LDS.
template <typename R, int THREADS, int CH, bool Q8>
__global__ __launch_bounds__(THREADS) void k_norm(mq_norm_args a, ScalesOut sc) {
  __shared__ float lds[2][THREADS / 64];
  const int64_t row = blockIdx.x;
  const int width = (int)a.width, tid = threadIdx.x;
  const float inv_w = 1.0f / (float)width;
  const _Float16* y = static_cast<const _Float16*>(a.y);
  const R* r = static_cast<const R*>(a.r) + row * a.r_stride;
  float v[CH][8], x[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int d = 8 * (c * THREADS + tid);
    if (y) take8(y + row * a.y_stride + d, width - d, x[c]);
    take8(r + d, width - d, v[c]);
  }
  if (y) {
    float scale = a.beta;
    if (a.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(x[c][i], x[c][i], s);
      s = sum_group<THREADS / 64>(s, lds[0]);
      scale = 1.0f / sqrtf(fmaf(s, inv_w, a.eps));
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int d = 8 * (c * THREADS + tid), left = width - d;
      float w[8];
      if (a.w_post) {
        take8(static_cast<const _Float16*>(a.w_post) + d, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * scale * (w[i] + a.weight_offset) * a.beta;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] *= scale;
      }
      if (a.gate) {
        take8(static_cast<const _Float16*>(a.gate) + row * a.gate_stride + d, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] *= w[i];
      }
      // the residual as it is stored: the next norm is taken from what a later reader finds
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = (float)(R)fp32(fmaf(a.alpha, v[c][i], x[c][i]));
      put8(static_cast<R*>(a.r_out) + row * a.r_out_stride + d, left, v[c]);
    }
  }
  if (!a.w_pre) return;
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(v[c][i], v[c][i], s);
  s = sum_group<THREADS / 64>(s, lds[1]);
  const float scale = 1.0f / sqrtf(fmaf(s, inv_w, a.eps));
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int d = 8 * (c * THREADS + tid), left = width - d;
    float w[8];
    take8(static_cast<const _Float16*>(a.w_pre) + d, left, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fp32(v[c][i] * scale * (w[i] + a.weight_offset));
    if constexpr (Q8) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= left) w[i] = 0.0f;   // also where the row's scale is NaN
        top = max(top, q8_magnitude(w[i]));
      }
      const uint32_t byte = q8_scale(q8_top16(top));
      const int first = d & ~(kQ8Block - 1);
      if (first < width) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.h_out) + row * a.h_stride + d) = q8_codes(w, byte);
        if (d == first) sc.p[row * sc.stride + d / kQ8Block] = (uint8_t)byte;
      }
    } else {
      put8(static_cast<_Float16*>(a.h_out) + row * a.h_stride + d, left, w);
    }
  }
}

// A launch takes fewer than 2^32 threads: more rows than that run in pieces of 2^31.
template <typename R, bool Q8, int THREADS, int CH>
hipError_t go(const mq_norm_args& a, const ScalesOut& sc, hipStream_t s) {
  constexpr int64_t step = (int64_t(1) << 31) / THREADS;
  for (int64_t t = 0; t < a.tokens; t += step) {
    mq_norm_args p = a;
    p.tokens = a.tokens - t < step ? a.tokens - t : step;
    if (a.y) p.y = static_cast<const _Float16*>(a.y) + t * a.y_stride;
    if (a.gate) p.gate = static_cast<const _Float16*>(a.gate) + t * a.gate_stride;
    p.r = static_cast<const R*>(a.r) + t * a.r_stride;
    if (a.y) p.r_out = static_cast<R*>(a.r_out) + t * a.r_out_stride;
    if (a.w_pre) p.h_out = static_cast<uint8_t*>(a.h_out) + t * a.h_stride * (Q8 ? 1 : 2);
    const ScalesOut q{Q8 ? sc.p + t * sc.stride : nullptr, sc.stride};
    k_norm<R, THREADS, CH, Q8><<<dim3((unsigned)p.tokens), dim3(THREADS), 0, s>>>(p, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename R, bool Q8>
hipError_t dispatch(const mq_norm_args& a, const ScalesOut& sc, hipStream_t s) {
  if (a.width <= 2048) return go<R, Q8, 256, 1>(a, sc, s);
  if (a.width <= 4096) return go<R, Q8, 512, 1>(a, sc, s);
  if (a.width <= 8192) return go<R, Q8, 1024, 1>(a, sc, s);
  if (a.width <= 16384) return go<R, Q8, 1024, 2>(a, sc, s);
  if (a.width <= 32768) return go<R, Q8, 1024, 4>(a, sc, s);
  return go<R, Q8, 1024, 8>(a, sc, s);
}

}  // namespace

hipError_t launch_norm_residual(const mq_norm_args& a, hipStream_t s) {
  return a.residual_fp32 ? dispatch<float, false>(a, {}, s) : dispatch<_Float16, false>(a, {}, s);
}

hipError_t launch_norm_residual_q8(const mq_norm_args& a, uint8_t* scales, int64_t scales_stride, hipStream_t s) {
  const ScalesOut sc{scales, scales_stride};
  return a.residual_fp32 ? dispatch<float, true>(a, sc, s) : dispatch<_Float16, true>(a, sc, s);
}

}  // namespace mq
