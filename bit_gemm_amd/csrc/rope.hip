// Rotary positions on their own (include/mosaicq_block.h, mq_rope) and their
// table.
//
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for each pair (a, b) of a head.
// Bound by HBM: 4 bytes an element (read and written once) and 8 bytes of
// table for each pair of a token, which all of its heads share. 8192 tokens of
// 64 heads of 128, half of each turned (271 MB): 50 us, 5.4 TB/s, the rate of a
// large copy. 16 tokens of 32 heads: 3.0 us, the launch and two dependent loads.
#include <algorithm>

#include "block_common.h"

namespace mq {
namespace {

// The frequencies come from the host in 64 bits, at most 512 of them, in the
// kernel's arguments; sine and cosine are taken in 64 bits and rounded once.
struct Freqs {
  double f[512];
};

__global__ __launch_bounds__(256) void k_rope_table(Freqs fr, int pairs, double mag, int64_t n,
                                                    float2* __restrict__ table) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= n) return;
  const int64_t p = idx / pairs;
  const int i = (int)(idx - p * pairs);
  double sn, cs;
  sincos((double)p * fr.f[i], &sn, &cs);
  table[idx] = make_float2((float)(cs * mag), (float)(sn * mag));
}

// A thread turns 8 pairs (half layout: two pieces of 8 elements rot / 2 apart) or 4 (interleaved: one piece) of HP heads
// of a token, which share the cosines and sines it loads once, or passes 8 elements on. Pieces lie where the head and
// the rotation put them, aligned or not; the last one of a kind may be shorter and goes element by element. A thread
// reads all that it turns before it writes, so y may be x.
template <int HP, bool INTER>
__global__ __launch_bounds__(256) void k_rope(const _Float16* x, uint32_t n, int heads, uint32_t units, int dim,
                                              int64_t xt, int64_t xh, const int32_t* __restrict__ pos, RopeView rope,
                                              float dir, _Float16* y, int64_t yt, int64_t yh) {
  const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
  if (idx >= n) return;
  const uint32_t hg = (uint32_t)(heads + HP - 1) / HP;
  const uint32_t row = idx / units;
  const int u = (int)(idx - row * units);
  const uint32_t t = row / hg;
  const int h0 = (int)(row - t * hg) * HP;
  const _Float16* xr = x + (int64_t)t * xt + h0 * xh;
  _Float16* yr = y + (int64_t)t * yt + h0 * yh;
  constexpr int NP = INTER ? 4 : 8;
  const int half = rope.rot >> 1, turns = (half + NP - 1) / NP;
  if (u >= turns) {
    const int d = rope.rot + 8 * (u - turns);
    if (d + 8 <= dim) {
      half8_t v[HP];
#pragma unroll
      for (int h = 0; h < HP; ++h)
        if (h0 + h < heads) v[h] = load8(xr + h * xh + d);
#pragma unroll
      for (int h = 0; h < HP; ++h)
        if (h0 + h < heads) store8(yr + h * yh + d, v[h]);
    } else {
      for (int h = 0; h < HP && h0 + h < heads; ++h)
        for (int e = d; e < dim; ++e) yr[h * yh + e] = xr[h * xh + e];
    }
    return;
  }
  const int i0 = NP * u, d = 8 * u;
  if (i0 + NP > half) {   // the last pairs
    for (int i = i0; i < half; ++i) {
      float2 cs = cos_sin(rope, pos[t], i);
      cs.y *= dir;
      const int a = INTER ? 2 * i : i, b = INTER ? a + 1 : i + half;
      for (int h = 0; h < HP && h0 + h < heads; ++h) {
        const float2 r = turn((float)xr[h * xh + a], (float)xr[h * xh + b], cs);
        yr[h * yh + a] = (_Float16)r.x;
        yr[h * yh + b] = (_Float16)r.y;
      }
    }
    return;
  }
  half8_t a[HP], b[HP];
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    if (h0 + h < heads) {
      a[h] = load8(xr + h * xh + d);
      if (!INTER) b[h] = load8(xr + h * xh + d + half);
    }
  }
  float2 cs[NP];
  load_cos_sin<NP>(rope, pos[t], i0, dir, cs);
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    if (h0 + h < heads) {
      turn_piece<INTER, NP>(a[h], b[h], cs);
      store8(yr + h * yh + d, a[h]);
      if (!INTER) store8(yr + h * yh + d + half, b[h]);
    }
  }
}

template <int HP>
void go(bool inter, int64_t n, const _Float16* x, int heads, int units, int dim, int64_t xt, int64_t xh,
        const int32_t* pos, const RopeView& rope, float dir, _Float16* y, int64_t yt, int64_t yh, hipStream_t s) {
  const dim3 g((unsigned)((n + 255) / 256)), b(256);
  if (inter)
    k_rope<HP, true><<<g, b, 0, s>>>(x, (uint32_t)n, heads, units, dim, xt, xh, pos, rope, dir, y, yt, yh);
  else
    k_rope<HP, false><<<g, b, 0, s>>>(x, (uint32_t)n, heads, units, dim, xt, xh, pos, rope, dir, y, yt, yh);
}

}  // namespace

hipError_t launch_rope_table(const double* freq, int pairs, double mag, int64_t positions, float2* table,
                             hipStream_t s) {
  Freqs fr;
  for (int i = 0; i < pairs; ++i) fr.f[i] = freq[i];
  for (int i = pairs; i < 512; ++i) fr.f[i] = 0.0;
  const int64_t n = positions * pairs;
  k_rope_table<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(fr, pairs, mag, n, table);
  return hipGetLastError();
}

hipError_t launch_rope(const _Float16* x, int64_t tokens, int heads, int dim, int64_t xt, int64_t xh,
                       const int32_t* pos, const RopeView& rope, int inverse, _Float16* y, int64_t yt, int64_t yh,
                       hipStream_t s) {
  const float dir = inverse ? -1.0f : 1.0f;
  const bool inter = rope.interleaved != 0;
  const int pairs = inter ? 4 : 8;
  const int units = (rope.rot / 2 + pairs - 1) / pairs + (dim - rope.rot + 7) / 8;
  // heads of a thread: 4 once that still leaves the GPU full (256 CUs of 1024 threads), else 1
  const int hp = tokens * heads * units >= 4 * 262144 ? 4 : 1;
  const int64_t per = (int64_t)((heads + hp - 1) / hp) * units;   // threads of a token
  // a launch covers fewer than 2^31 threads: more tokens than that run in pieces
  const int64_t step = std::max<int64_t>(1, ((int64_t(1) << 31) - 1) / per);
  for (int64_t t = 0; t < tokens; t += step) {
    const int64_t n = std::min(step, tokens - t) * per;
    if (hp == 4)
      go<4>(inter, n, x + t * xt, heads, units, dim, xt, xh, pos + t, rope, dir, y + t * yt, yt, yh, s);
    else
      go<1>(inter, n, x + t * xt, heads, units, dim, xt, xh, pos + t, rope, dir, y + t * yt, yt, yh, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mq
