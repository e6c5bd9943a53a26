// Rotary positions on their own (include/mosaicq_block.h, mq_rope) and their
// table.
//
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for each pair (a, b) of a head.
// Bound by HBM: 4 bytes an element (read and written once) and 8 bytes of
// table for each pair of a token, which all of its heads share.
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

// One thread for each pair, and for each element that passes: any size, stride
// or alignment. A thread reads both elements of its pair before it writes, so
// y may be x.
__global__ __launch_bounds__(256) void k_rope_any(const _Float16* x, int64_t n, int heads, int units, int dim,
                                                  int64_t xt, int64_t xh, const int32_t* __restrict__ pos,
                                                  RopeView rope, float dir, _Float16* y, int64_t yt, int64_t yh) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= n) return;
  const int64_t row = idx / units;
  const int u = (int)(idx - row * units);
  const int64_t t = row / heads;
  const int h = (int)(row - t * heads);
  const _Float16* xr = x + t * xt + h * xh;
  _Float16* yr = y + t * yt + h * yh;
  const int pairs = rope.rot >> 1;
  if (u >= pairs) {
    yr[rope.rot + u - pairs] = xr[rope.rot + u - pairs];
    return;
  }
  const int a = rope.interleaved ? 2 * u : u, b = rope.interleaved ? a + 1 : u + pairs;
  float2 cs = cos_sin(rope, pos[t], u);
  cs.y *= dir;
  const float2 r = turn((float)xr[a], (float)xr[b], cs);
  yr[a] = (_Float16)r.x;
  yr[b] = (_Float16)r.y;
}

// The same in 16-byte pieces: a thread turns 8 pairs (half layout: two pieces
// rot / 2 apart) or 4 (interleaved: one piece) of HP heads of a token, which
// share the cosines and sines it loads once.
template <int HP, bool INTER>
__global__ __launch_bounds__(256) void k_rope_vec(const _Float16* x, uint32_t n, int heads, uint32_t units, int dim,
                                                  int64_t xt, int64_t xh, const int32_t* __restrict__ pos,
                                                  RopeView rope, float dir, _Float16* y, int64_t yt, int64_t yh) {
  const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
  if (idx >= n) return;
  const uint32_t hg = (uint32_t)(heads + HP - 1) / HP;
  const uint32_t row = idx / units;
  const int u = (int)(idx - row * units);
  const uint32_t t = row / hg;
  const int h0 = (int)(row - t * hg) * HP;
  const _Float16* xr = x + (int64_t)t * xt + h0 * xh;
  _Float16* yr = y + (int64_t)t * yt + h0 * yh;
  const int half = rope.rot >> 1;
  const int turn_units = INTER ? rope.rot >> 3 : rope.rot >> 4;
  if (u >= turn_units) {
    const int d = rope.rot + 8 * (u - turn_units);
    half8_t v[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h)
      if (h0 + h < heads) v[h] = *reinterpret_cast<const half8_t*>(xr + h * xh + d);
#pragma unroll
    for (int h = 0; h < HP; ++h)
      if (h0 + h < heads) *reinterpret_cast<half8_t*>(yr + h * yh + d) = v[h];
    return;
  }
  constexpr int NP = INTER ? 4 : 8;
  half8_t a[HP], b[HP];
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    if (h0 + h < heads) {
      a[h] = *reinterpret_cast<const half8_t*>(xr + h * xh + 8 * u);
      if (!INTER) b[h] = *reinterpret_cast<const half8_t*>(xr + h * xh + 8 * u + half);
    }
  }
  float2 cs[NP];
  load_cos_sin<NP>(rope, pos[t], NP * u, dir, cs);
#pragma unroll
  for (int h = 0; h < HP; ++h) {
    if (h0 + h < heads) {
      turn_piece<INTER, NP>(a[h], b[h], cs);
      *reinterpret_cast<half8_t*>(yr + h * yh + 8 * u) = a[h];
      if (!INTER) *reinterpret_cast<half8_t*>(yr + h * yh + 8 * u + half) = b[h];
    }
  }
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
  if (tokens == 0) return hipSuccess;
  const float dir = inverse ? -1.0f : 1.0f;
  const bool inter = rope.interleaved != 0;
  const int piece = inter ? 8 : 16;   // rotated elements of a unit
  const int units = rope.rot / piece + (dim - rope.rot) / 8;
  // heads of a thread: 4 once that still leaves the GPU full (256 CUs of 1024 threads), else 1
  const int64_t one = tokens * heads * units;
  const int hp = one >= 4 * 262144 ? 4 : 1;
  const int64_t n = tokens * ((heads + hp - 1) / hp) * units;
  if (piecewise(rope) && dim % 8 == 0 && wide_rows(x, xt) && xh % 8 == 0 && wide_rows(y, yt) && yh % 8 == 0 &&
      n < (int64_t(1) << 31)) {
    const dim3 g((unsigned)((n + 255) / 256)), b(256);
    const uint32_t un = (uint32_t)n, uu = (uint32_t)units;
    if (inter) {
      if (hp == 4)
        k_rope_vec<4, true><<<g, b, 0, s>>>(x, un, heads, uu, dim, xt, xh, pos, rope, dir, y, yt, yh);
      else
        k_rope_vec<1, true><<<g, b, 0, s>>>(x, un, heads, uu, dim, xt, xh, pos, rope, dir, y, yt, yh);
    } else {
      if (hp == 4)
        k_rope_vec<4, false><<<g, b, 0, s>>>(x, un, heads, uu, dim, xt, xh, pos, rope, dir, y, yt, yh);
      else
        k_rope_vec<1, false><<<g, b, 0, s>>>(x, un, heads, uu, dim, xt, xh, pos, rope, dir, y, yt, yh);
    }
    return hipGetLastError();
  }
  // one launch covers at most 2^31 - 1 workgroups of 256 units: more tokens than that run in pieces
  const int any = rope.rot / 2 + dim - rope.rot;
  const int64_t step = ((int64_t(1) << 38) / ((int64_t)heads * any));
  for (int64_t t = 0; t < tokens; t += step) {
    const int64_t m = (tokens - t < step ? tokens - t : step) * heads * any;
    k_rope_any<<<dim3((unsigned)((m + 255) / 256)), dim3(256), 0, s>>>(x + t * xt, m, heads, any, dim, xt, xh, pos + t,
                                                                      rope, dir, y + t * yt, yt, yh);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mq
