// Norms before and after a block with its gate and residual
// (include/mosaicq_block.h, mq_norm_residual).
//
//   r' = alpha r + beta g (y / rms(y)) (w_post + o),  h = (r' / rms(r')) (w_pre + o)
//
// One workgroup a row, the row in registers from the first read to the last
// write, so every input is read once; two sums over the row, of y^2 and of
// r'^2, in fp32, a thread's own elements first, then the lanes of a wave, then
// the waves in order. Bound by HBM for many rows (y, r, gate read, r', h
// written); by the two dependent sums and the load before them for few.
#include "block_common.h"

namespace mq {
namespace {

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

// 8 elements from p (or those of them below `left`, one by one, where the
// rows do not allow 16-byte accesses or end inside the piece).
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* p, int left, float* v) {
  if (VEC) {
    if (left > 0) {
      if (sizeof(T) == 2) {
        const half8_t h = *reinterpret_cast<const half8_t*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
      } else {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? (float)p[i] : 0.0f;
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int left, const float* v) {
  if (VEC) {
    if (left > 0) {
      if (sizeof(T) == 2) {
        half8_t h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
        *reinterpret_cast<half8_t*>(p) = h;
      } else {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (T)v[i];
  }
}

// CH pieces of 8 elements a thread. Multiply-adds are written out, so that
// both forms of access give the same bits.
template <typename R, bool VEC, int THREADS, int CH>
__global__ __launch_bounds__(THREADS) void k_norm(mq_norm_args a) {
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
    if (y) load8<VEC>(y + row * a.y_stride + d, width - d, x[c]);
    load8<VEC>(r + d, width - d, v[c]);
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
        load8<VEC>(static_cast<const _Float16*>(a.w_post) + d, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * scale * (w[i] + a.weight_offset) * a.beta;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] *= scale;
      }
      if (a.gate) {
        load8<VEC>(static_cast<const _Float16*>(a.gate) + row * a.gate_stride + d, left, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[c][i] *= w[i];
      }
      // the residual as it is stored: the next norm is taken from what a later reader finds
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = (float)(R)fp32(fmaf(a.alpha, v[c][i], x[c][i]));
      store8<VEC>(static_cast<R*>(a.r_out) + row * a.r_out_stride + d, left, v[c]);
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
    load8<VEC>(static_cast<const _Float16*>(a.w_pre) + d, left, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fp32(v[c][i] * scale * (w[i] + a.weight_offset));
    store8<VEC>(static_cast<_Float16*>(a.h_out) + row * a.h_stride + d, left, w);
  }
}

template <typename R, bool VEC>
void dispatch(const mq_norm_args& a, hipStream_t s) {
  const dim3 g((unsigned)a.tokens);
  if (a.width <= 2048)
    k_norm<R, VEC, 256, 1><<<g, dim3(256), 0, s>>>(a);
  else if (a.width <= 4096)
    k_norm<R, VEC, 512, 1><<<g, dim3(512), 0, s>>>(a);
  else if (a.width <= 8192)
    k_norm<R, VEC, 1024, 1><<<g, dim3(1024), 0, s>>>(a);
  else if (a.width <= 16384)
    k_norm<R, VEC, 1024, 2><<<g, dim3(1024), 0, s>>>(a);
  else if (a.width <= 32768)
    k_norm<R, VEC, 1024, 4><<<g, dim3(1024), 0, s>>>(a);
  else
    k_norm<R, VEC, 1024, 8><<<g, dim3(1024), 0, s>>>(a);
}

}  // namespace

hipError_t launch_norm_residual(const mq_norm_args& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  // 16-byte accesses where every row of every array allows them
  const auto wide = [&](const void* p, int64_t stride, int size) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * size) % 16 == 0);
  };
  const int rs = a.residual_fp32 ? 4 : 2;
  const bool vec = a.width % 8 == 0 && wide(a.y, a.y_stride, 2) && wide(a.r, a.r_stride, rs) &&
                   wide(a.gate, a.gate_stride, 2) && wide(a.w_post, 0, 2) && wide(a.w_pre, 0, 2) &&
                   wide(a.y ? a.r_out : nullptr, a.r_out_stride, rs) && wide(a.w_pre ? a.h_out : nullptr, a.h_stride, 2);
  if (a.residual_fp32) {
    if (vec) dispatch<float, true>(a, s); else dispatch<float, false>(a, s);
  } else {
    if (vec) dispatch<_Float16, true>(a, s); else dispatch<_Float16, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace mq
