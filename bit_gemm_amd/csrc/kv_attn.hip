// Attention over the 8-bit key/value cache (include/mosaicq_block.h,
// mq_kv_attention), for few query rows: single tokens and short pieces.
//
// A kv head's query rows are its n new tokens times the g query heads that
// share it, row r = token r / g, head r % g. A workgroup of 4 waves holds
// 16 NT rows and a chunk of the sequence's 64-token cache blocks; its waves
// take the blocks in turn, each with its own running maximum m and sum l:
//   S^T = K Q^T        16x16x32 fp16 MFMA, keys as the A operand: lane
//                      (c = l % 16, g = l / 16) of tile t gets the scores of
//                      row c and tokens 16 g + 4 t + 0..3 if tile row R holds
//                      token 16 (R / 4) + 4 t + R % 4;
//   P = 2^(S - m)      in that layout lane g holds tokens 16 g .. 16 g + 15:
//                      just the B operand of the next product, without LDS;
//   O^T += V^T P^T     values lie transposed in the cache, so a lane's 16
//                      bytes are 16 tokens of one element: again the A operand.
// Codes become fp16 in registers (exactly: int8 and e4m3 values are fp16
// values); a block's scales multiply the fp32 scores and the fp32 product.
// P is rounded to fp16 (relative 2^-11, and the sum l takes the unrounded
// values); everything else is fp32.
//
// The waves' results are joined in LDS in wave order. Where the sequences do
// not fill the GPU, the cache is split over workgroups, whose partial results
// go to the workspace and are joined in split order by k_attn_join.
// Bound by HBM: 2 head_dim bytes for each cached token and kv head.
#include <algorithm>

#include "kv_attn_common.h"

namespace mq {
namespace {

// The largest of the four lanes that share l % 16, in all of them.
__device__ __forceinline__ float max_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// One block's keys and values in registers, as codes or (open block) as fp16.
template <int D>
struct Codes {
  uint4 k[4][D / 64], v[D / 16];
};

template <int D, int FMT, int NT>
__global__ __launch_bounds__(256) void k_attn_split(AttnArgs A) {
  constexpr int DT = D / 16, KS = D / 32;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  // workgroup -> (sequence, row tile, kv head, split)
  int w = (int)blockIdx.x;
  const int split = w % A.splits;
  w /= A.splits;
  const int h = w % A.kv.hk;
  w /= A.kv.hk;
  const int rt = w % A.row_tiles, s = w / A.row_tiles;
  const Seq sq = seq_of(A.b, A.kv, s);
  const int rows = sq.n * A.group, row0 = rt * 16 * NT;
  if (row0 >= rows) return;
  const int len = sq.cap;

  // this lane's rows: where they end, and their queries as the B operand
  int end[NT], last = 0, first_end = len;
  half8_t qf[NT][KS];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = row0 + 16 * t + c;
    const int rr = r < rows ? r : row0;
    const int tok = rr / A.group, hh = rr % A.group;
    const _Float16* qp = A.q.p + (int64_t)(sq.q0 + tok) * A.q.stride + (int64_t)(h * A.group + hh) * D;
#pragma unroll
    for (int j = 0; j < D / 64; ++j)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        qf[t][2 * j + x] = *reinterpret_cast<const half8_t*>(qp + 64 * j + 16 * g + 8 * x);
    const int e = A.causal ? max(len - sq.n + tok + 1, 0) : len;
    end[t] = r < rows ? e : 0;
    last = max(last, end[t]);
    first_end = min(first_end, e);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    last = max(last, __shfl_xor(last, d));
    first_end = min(first_end, __shfl_xor(first_end, d));
  }
  last = __builtin_amdgcn_readfirstlane(last);
  first_end = __builtin_amdgcn_readfirstlane(first_end);

  const int nblk = (last + kKvBlock - 1) / kKvBlock;
  const int b0 = split * A.chunk, b1 = min(nblk, b0 + A.chunk);
  const int open_blk = len / kKvBlock;

  float4_t o[NT][DT];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (int b = b0 + wave; b < b1; b += 4) {
    half8_t vf[DT][2];
    float4_t sc[NT][4];
    float ks, vs;
    const int ktok = 16 * (c >> 2) + (c & 3);   // + 4 t: the token of this lane's row of key tile t
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[t][k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
    if (b != open_blk) {
      const int id0 = A.b.table[(int64_t)s * A.b.width + b];
      const bool ok = (uint64_t)(int64_t)id0 < (uint64_t)A.kv.blocks;
      const int64_t head = (int64_t)(ok ? id0 : 0) * A.kv.hk + h;
      ks = ok ? A.kv.ks[head] : __builtin_nanf("");
      vs = A.kv.vs[head];
      const uint8_t* kp = A.kv.kc + head * (kKvBlock * D);
      const uint8_t* vp = A.kv.vc + head * (kKvBlock * D);
      Codes<D> cd;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
          cd.k[k][j] = *reinterpret_cast<const uint4*>(kp + (ktok + 4 * k) * D + 64 * j + 16 * g);
#pragma unroll
      for (int d = 0; d < DT; ++d)
        cd.v[d] = *reinterpret_cast<const uint4*>(vp + (16 * d + c) * kKvBlock + 16 * g);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          const half8_t a0 = widen8<FMT>(cd.k[k][j].x, cd.k[k][j].y), a1 = widen8<FMT>(cd.k[k][j].z, cd.k[k][j].w);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            sc[t][k] = mfma16(a0, qf[t][2 * j], sc[t][k]);
            sc[t][k] = mfma16(a1, qf[t][2 * j + 1], sc[t][k]);
          }
        }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        vf[d][0] = widen8<FMT>(cd.v[d].x, cd.v[d].y);
        vf[d][1] = widen8<FMT>(cd.v[d].z, cd.v[d].w);
      }
    } else {
      // the open block: fp16 in the sequence's tail, tokens from `left` on are not the sequence's
      const int left = len - b * kKvBlock;
      ks = sq.slot >= 0 ? 1.0f : __builtin_nanf("");
      vs = 1.0f;
      const int64_t head = ((int64_t)max(sq.slot, 0) * A.kv.hk + h) * (kKvBlock * D);
      const _Float16* kp = A.kv.kt + head;
      const _Float16* vp = A.kv.vt + head;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const half8_t a = *reinterpret_cast<const half8_t*>(kp + (ktok + 4 * k) * D + 64 * j + 16 * g + 8 * x);
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][k] = mfma16(a, qf[t][2 * j + x], sc[t][k]);
          }
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          half8_t a = *reinterpret_cast<const half8_t*>(vp + (16 * d + c) * kKvBlock + 16 * g + 8 * x);
#pragma unroll
          for (int i = 0; i < 8; ++i)   // whatever stands past the end may be no number: 0 x it is kept out
            if (16 * g + 8 * x + i >= left) a[i] = (_Float16)0.0f;
          vf[d][x] = a;
        }
    }
    const float f = ks * A.scale2;
    const bool masked = (b + 1) * kKvBlock > first_end;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = -INFINITY;
      float p[16];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = sc[t][k][i] * f;
          if (masked && b * kKvBlock + 16 * g + 4 * k + i >= end[t]) v = -INFINITY;
          p[4 * k + i] = v;
          top = fmaxf(top, v);
        }
      top = fmaxf(m[t], max_groups(top));
      const float ref = top == -INFINITY ? 0.0f : top;
      const float shrink = __builtin_amdgcn_exp2f(m[t] - ref);
      m[t] = top;
      float sum = 0.0f;
      half8_t pf[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = __builtin_amdgcn_exp2f(p[i] - ref);
        sum += e;
        pf[i >> 3][i & 7] = (_Float16)e;
      }
      l[t] = l[t] * shrink + sum;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        float4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
        a = mfma16(vf[d][0], pf[0], a);
        a = mfma16(vf[d][1], pf[1], a);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][d][i] = o[t][d][i] * shrink + a[i] * vs;
      }
    }
  }

  // join the waves
  __shared__ float sm[4][16 * NT], sl[4][16 * NT];
  __shared__ float so[16 * NT][D + 4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] = sum_groups(l[t]);
    if (g == 0) {
      sm[wave][16 * t + c] = m[t];
      sl[wave][16 * t + c] = l[t];
    }
  }
  __syncthreads();
  float top[NT], total[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 16 * t + c;
    top[t] = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
    const float ref = top[t] == -INFINITY ? 0.0f : top[t];
    total[t] = 0.0f;
#pragma unroll
    for (int x = 0; x < 4; ++x) total[t] += sl[x][r] * __builtin_amdgcn_exp2f(sm[x][r] - ref);
    const float f = __builtin_amdgcn_exp2f(m[t] - ref);
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d] *= f;
  }
  for (int x = 0; x < 4; ++x) {   // wave by wave: the sum's order is fixed
    if (wave == x) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          float4_t* p = reinterpret_cast<float4_t*>(&so[16 * t + c][16 * d + 4 * g]);
          *p = x == 0 ? o[t][d] : *p + o[t][d];
        }
    }
    __syncthreads();
  }
  if (wave == 0 && g == 0) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sm[0][16 * t + c] = top[t];
      sl[0][16 * t + c] = total[t];
    }
  }
  __syncthreads();
  for (int e = tid; e < 16 * NT * (D / 4); e += 256) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    if (row0 + r >= rows) break;
    const int tok = (row0 + r) / A.group, hh = (row0 + r) % A.group;
    const int64_t row = (int64_t)(sq.q0 + tok) * A.hq + h * A.group + hh;
    const float4_t v = *reinterpret_cast<const float4_t*>(&so[r][d]);
    if (A.splits == 1) {
      const float inv = sl[0][r] == 0.0f ? 0.0f : 1.0f / sl[0][r];
      store4(reinterpret_cast<uint16_t*>(A.out.p + (int64_t)(sq.q0 + tok) * A.out.stride + (int64_t)(h * A.group + hh) * D + d),
             v * inv, 4, true);
    } else {
      *reinterpret_cast<float4_t*>(A.ws_o + (row * A.splits + split) * D + d) = v;
      if (d == 0) A.ws_ml[row * A.splits + split] = make_float2(sm[0][r], sl[0][r]);
    }
  }
}

// Joins the splits of one (token, query head) row in split order: one wave a row.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs A, int64_t rows) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const float2* ml = A.ws_ml + row * A.splits;
  float top = -INFINITY;
  for (int x = lane; x < A.splits; x += 64) top = fmaxf(top, ml[x].x);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == -INFINITY ? 0.0f : top;
  float acc[D / 64], total = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) acc[i] = 0.0f;
  for (int x = 0; x < A.splits; ++x) {
    const float2 v = ml[x];
    const float f = __builtin_amdgcn_exp2f(v.x - ref);
    total += v.y * f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) acc[i] += A.ws_o[(row * A.splits + x) * D + lane + 64 * i] * f;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t tok = row / A.hq, hh = row % A.hq;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) A.out.p[tok * A.out.stride + hh * D + lane + 64 * i] = (_Float16)(acc[i] * inv);
}

template <int D, int FMT>
hipError_t go(const AttnArgs& A, const AttnPlan& p, hipStream_t s) {
  const dim3 g((unsigned)p.groups), t(256);
  hipError_t e = hipSuccess;
  if (p.nt == 0) {
    e = launch_attn_rows(A, D, FMT, p, s);
  } else {
    switch (p.nt) {
      case 1: k_attn_split<D, FMT, 1><<<g, t, 0, s>>>(A); break;
      case 2: k_attn_split<D, FMT, 2><<<g, t, 0, s>>>(A); break;
      default: k_attn_split<D, FMT, 4><<<g, t, 0, s>>>(A); break;
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)A.b.tokens * A.hq;
  k_attn_join<D><<<dim3((unsigned)((rows + 3) / 4)), t, 0, s>>>(A, rows);
  return hipGetLastError();
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

AttnPlan plan_attention(int hk, int hq, int dim, int64_t seqs, int64_t tokens, int64_t max_new, int64_t max_len) {
  AttnPlan p{};
  if (max_new > tokens && tokens > 0) max_new = tokens;
  const int64_t rows = max_new * (hq / hk), blocks = up(max_len, kKvBlock);
  int64_t one, splits;
  if (rows <= 64) {
    p.nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    // split the cache until the GPU has about 4 workgroups a CU, but leave a wave at least two blocks
    p.row_tiles = (int)up(rows, 16 * p.nt);
    one = seqs * p.row_tiles * hk;
    splits = one > 0 ? std::min(up(1024, one), up(blocks, 8)) : 1;
  } else {
    // split the cache, 16 blocks at least a part, until there are about two workgroups a CU (as far as
    // the host can tell: the tokens give the row tiles that there are, where sequences differ in length)
    p.row_tiles = (int)up(rows, kAttnRows);
    one = seqs * p.row_tiles * hk;
    const int64_t tiles = std::min(seqs * p.row_tiles, tokens * (hq / hk) / kAttnRows + seqs);
    splits = one > 0 ? std::min(up(512, tiles * hk), up(blocks, 16)) : 1;
  }
  if (splits > 256) splits = 256;
  p.chunk = (int)up(blocks, splits);
  p.splits = (int)up(blocks, p.chunk);
  p.groups = one * p.splits;
  p.bytes = p.splits == 1 ? 0 : (size_t)(tokens * hq) * p.splits * ((size_t)dim * 4 + 8);
  return p;
}

hipError_t launch_kv_attention(const KvView& kv, int dim, int format, const BatchView& b, RowsIn q, int hq, int causal,
                               float scale, RowsOut out, void* ws, const AttnPlan& plan, hipStream_t s) {
  if (plan.groups == 0 || b.tokens == 0) return hipSuccess;
  AttnArgs A;
  A.kv = kv;
  A.b = b;
  A.q = q;
  A.out = out;
  A.hq = hq;
  A.group = hq / kv.hk;
  A.causal = causal;
  A.scale2 = scale * kLog2e;
  A.row_tiles = plan.row_tiles;
  A.chunk = plan.chunk;
  A.splits = plan.splits;
  A.ws_o = static_cast<float*>(ws);
  A.ws_ml = reinterpret_cast<float2*>(A.ws_o + (size_t)b.tokens * hq * plan.splits * dim);
  if (dim == 64)
    return format == MQ_KV_INT8 ? go<64, MQ_KV_INT8>(A, plan, s) : go<64, MQ_KV_E4M3>(A, plan, s);
  return format == MQ_KV_INT8 ? go<128, MQ_KV_INT8>(A, plan, s) : go<128, MQ_KV_E4M3>(A, plan, s);
}

}  // namespace mq
