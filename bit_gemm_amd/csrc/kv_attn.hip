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
// values). A block's scales stay in fp32: with t = (k scale) s + log2(v scale)
// the weights are p = 2^(t - m), so that O sums codes in units of 2^-m and no
// block needs its own accumulator; the softmax's sum takes p / (v scale). p is
// rounded to fp16 (relative 2^-11, down to 2^-29 of the largest: m lies 15 below
// the largest t); its sum is not, since a block of small values has small p
// whatever its scores. All else is fp32.
//
// Bound by HBM: 2 head_dim bytes for each cached token and kv head. A wave's
// loads are never conditional and keys of its next block are requested as soon
// as this block's are multiplied, values likewise, so something is in flight
// at all times; registers for two waves a SIMD.
// The waves' results are joined in LDS in wave order. Where the sequences do
// not fill the GPU, the cache is split over workgroups, whose partial results
// go to the workspace and are joined in a fixed order by k_attn_join.
// Heads of 128: 16 tokens of 500 to 4096 cached ones, 32 kv heads (282 MB): 51 us,
// 5.5 TB/s; 2 of 65500, 8 kv heads (267 MB): 41 us, 6.5 TB/s, and 4.7 us to join;
// one of 300: 8 us, of which 4 are the launch and the chain of its loads.
#include <algorithm>

#include "kv_attn_common.h"

namespace mq {
namespace {

constexpr int kWaves = 4;   // of a workgroup of k_attn_split

// The largest of the four lanes that share l % 16, in all of them.
__device__ __forceinline__ float max_groups(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <int D, int FMT, int NT>
__global__ __launch_bounds__(64 * kWaves, NT == 4 ? 1 : 2) void k_attn_split(AttnArgs A) {
  constexpr int DT = D / 16, KS = D / 32;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15, g = lane >> 4;
  // workgroup -> (sequence, row tile, split, kv head)
  int w = (int)blockIdx.x;
  const int h = w % A.kv.hk;
  w /= A.kv.hk;
  const int split = w % A.splits;
  w /= A.splits;
  const int rt = w % A.row_tiles, s = w / A.row_tiles;
  // this wave's blocks: bw, bw + kWaves, ... Numbers and codes are requested whether the block exists and is coded or not
  // (in its place one that does), so that nothing waits for them before they are used.
  const int bw = split * A.chunk + wave, table_last = A.b.width - 1;
  const uint32_t blocks = (uint32_t)A.kv.blocks;
  const int32_t* table = A.b.table + (int64_t)s * A.b.width;
  const auto id_of = [&](int b) { return table[min(b, table_last)]; };
  const auto head_of = [&](int id) { return (int64_t)((uint32_t)id < blocks ? id : 0) * A.kv.hk + h; };
  int id = id_of(bw), id_1 = id_of(bw + kWaves);
  const Seq sq = seq_of(A.b, A.kv, s);
  const int rows = sq.n * A.group, row0 = rt * 16 * NT;
  if (row0 >= rows) return;
  const int len = sq.cap;

  const int ktok = 16 * (c >> 2) + (c & 3);   // + 4 k: the token of this lane's row of key tile k
  uint4 kc[4][D / 64], vc[DT];
  const auto load_keys = [&](int id) {
    const uint8_t* p = A.kv.kc + head_of(id) * (kKvBlock * D) + ktok * D + 16 * g;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < D / 64; ++j) kc[k][j] = *reinterpret_cast<const uint4*>(p + 4 * k * D + 64 * j);
  };
  const auto load_values = [&](int id) {
    const uint8_t* p = A.kv.vc + head_of(id) * (kKvBlock * D) + c * kKvBlock + 16 * g;
#pragma unroll
    for (int d = 0; d < DT; ++d) vc[d] = *reinterpret_cast<const uint4*>(p + 16 * d * kKvBlock);
  };
  load_keys(id);
  load_values(id);
  float ks = A.kv.ks[head_of(id)], vs = A.kv.vs[head_of(id)];   // of this block, as loaded, a turn ahead

  // this lane's rows: where they end, and their queries as the B operand
  int end[NT];
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
    end[t] = r >= rows ? 0 : A.causal ? max(len - sq.n + tok + 1, 0) : len;
  }
  // rows see more the later they are: the last one says how far, the first how far all see
  const int last_row = min(rows, row0 + 16 * NT) - 1;
  const int last = A.causal ? max(len - sq.n + last_row / A.group + 1, 0) : len;
  const int all = A.causal ? max(len - sq.n + row0 / A.group + 1, 0) : len;
  const int nblk = (last + kKvBlock - 1) / kKvBlock, open_blk = len / kKvBlock;
  const int b1 = min(nblk, (split + 1) * A.chunk), coded = min(b1, open_blk);

  float4_t o[NT][DT];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = kNoMax;
    l[t] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[t][d] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  }
  float4_t sc[NT][4];
  half8_t pf[NT][2];
  // The weights of block b from its scores: sc[t][k][i] is row 16 t + c, token 16 g + 4 k + i.
  const auto weights = [&](int b, float ks, float vs) {
    vs = vs == 0.0f ? kZeroScale : vs;
    const float mul = ks * A.scale2, add = __builtin_amdgcn_logf(vs);
    const bool masked = (b + 1) * kKvBlock > all;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int left = end[t] - b * kKvBlock - 16 * g;
      float p[16], top = kNoMax;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = fmaf(sc[t][i >> 2][i & 3], mul, add);
        if (masked && i >= left) p[i] = -INFINITY;
        top = fmaxf(top, p[i]);
      }
      top = reference(max_groups(top), kMaxWeight);
      if (__any(top > m[t])) {
        const float now = fmaxf(m[t], top), shrink = __builtin_amdgcn_exp2f(m[t] - now);
        m[t] = now;
        l[t] *= shrink;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[t][d] *= shrink;
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = __builtin_amdgcn_exp2f(p[i] - m[t]);
        sum += e;
        pf[t][i >> 3][i & 7] = (_Float16)e;
      }
      l[t] = fmaf(sum, __builtin_amdgcn_rcpf(vs), l[t]);
    }
  };
  const auto no_scores = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[t][k] = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
  };

  if (bw + kWaves >= coded) id_1 = id;   // past its last coded block a wave requests that one again: it is near
  int b = bw;
  for (; b < coded; b += kWaves) {
    no_scores();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const half8_t a0 = widen8<FMT>(kc[k][j].x, kc[k][j].y), a1 = widen8<FMT>(kc[k][j].z, kc[k][j].w);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          sc[t][k] = mfma16(a0, qf[t][2 * j], sc[t][k]);
          sc[t][k] = mfma16(a1, qf[t][2 * j + 1], sc[t][k]);
        }
      }
    load_keys(id_1);
    const float k1 = (uint32_t)id < blocks ? ks : __builtin_nanf(""), v1 = vs;
    ks = A.kv.ks[head_of(id_1)];
    vs = A.kv.vs[head_of(id_1)];
    const int id_2 = b + 2 * kWaves < coded ? id_of(b + 2 * kWaves) : id_1;
    weights(b, k1, v1);
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const half8_t a0 = widen8<FMT>(vc[d].x, vc[d].y), a1 = widen8<FMT>(vc[d].z, vc[d].w);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][d] = mfma16(a0, pf[t][0], o[t][d]);
        o[t][d] = mfma16(a1, pf[t][1], o[t][d]);
      }
    }
    load_values(id_1);
    id = id_1;
    id_1 = id_2;
  }
  if (b == open_blk && b < b1) {
    // the open block: fp16 in the sequence's tail; tokens from `left` on are not the sequence's and may be no numbers
    const int left = len - b * kKvBlock;
    const int64_t head = ((int64_t)max(sq.slot, 0) * A.kv.hk + h) * (kKvBlock * D);
    const _Float16* kp = A.kv.kt + head + ktok * D + 16 * g;
    const _Float16* vp = A.kv.vt + head + c * kKvBlock + 16 * g;
    no_scores();
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const half8_t a = *reinterpret_cast<const half8_t*>(kp + 4 * k * D + 64 * j + 8 * x);
#pragma unroll
          for (int t = 0; t < NT; ++t) sc[t][k] = mfma16(a, qf[t][2 * j + x], sc[t][k]);
        }
    weights(b, sq.slot >= 0 ? 1.0f : __builtin_nanf(""), 1.0f);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        half8_t a = *reinterpret_cast<const half8_t*>(vp + 16 * d * kKvBlock + 8 * x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (16 * g + 8 * x + i >= left) a[i] = (_Float16)0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t][d] = mfma16(a, pf[t][x], o[t][d]);
      }
  }

  // join the waves
  // few rows: every wave's sums side by side, added as they are written out; else one after the other into one place
  constexpr int SIDES = NT == 1 ? kWaves : 1;
  __shared__ float sm[kWaves][16 * NT], sl[kWaves][16 * NT];
  __shared__ float so[SIDES][16 * NT][D + 4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (end[t] > 0) l[t] += zero_if_finite(qf[t]);
    l[t] = sum_groups(l[t]);
    if (g == 0) {
      sm[wave][16 * t + c] = m[t];
      sl[wave][16 * t + c] = l[t];
    }
  }
  __syncthreads();
  const auto top_of = [&](int r) {
    float top = sm[0][r];
#pragma unroll
    for (int x = 1; x < kWaves; ++x) top = fmaxf(top, sm[x][r]);
    return top;
  };
  for (int x = SIDES == 1 ? 0 : wave; x < (SIDES == 1 ? kWaves : wave + 1); ++x) {   // wave by wave: the sum's order is fixed
    if (wave == x) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float f = __builtin_amdgcn_exp2f(m[t] - top_of(16 * t + c));
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          float4_t* p = reinterpret_cast<float4_t*>(&so[SIDES == 1 ? 0 : wave][16 * t + c][16 * d + 4 * g]);
          *p = SIDES > 1 || x == 0 ? o[t][d] * f : *p + o[t][d] * f;
        }
      }
    }
    if (SIDES == 1) __syncthreads();
  }
  if (SIDES > 1) __syncthreads();
  for (int e = tid; e < 16 * NT * (D / 4); e += 64 * kWaves) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    if (row0 + r >= rows) break;
    const int tok = (row0 + r) / A.group, hh = (row0 + r) % A.group;
    const int64_t row = (int64_t)(sq.q0 + tok) * A.hq + h * A.group + hh;
    float4_t v = *reinterpret_cast<const float4_t*>(&so[0][r][d]);
#pragma unroll
    for (int x = 1; x < SIDES; ++x) v += *reinterpret_cast<const float4_t*>(&so[x][r][d]);
    const float top = top_of(r);
    float total = 0.0f;
#pragma unroll
    for (int x = 0; x < kWaves; ++x) total += sl[x][r] * __builtin_amdgcn_exp2f(sm[x][r] - top);
    if (A.splits == 1) {
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      store4(reinterpret_cast<uint16_t*>(A.out.p + (int64_t)(sq.q0 + tok) * A.out.stride + (int64_t)(h * A.group + hh) * D + d),
             v * inv, 4, true);
    } else {
      *reinterpret_cast<float4_t*>(A.ws_o + (row * A.splits + split) * D + d) = v;
      if (d == 0) A.ws_ml[row * A.splits + split] = make_float2(top, total);
    }
  }
}

// Joins the splits of (token, query head) rows: Y groups of threads a row, group y takes splits y, y + Y, ...; in a
// group thread x takes elements 4 x .. 4 x + 3. The groups' sums are added in order. One group a row where the splits
// are few and the rows many, else all of the workgroup's. Rows of no sequence have no partial results: what
// is read for them is not looked at.
template <int D, int Y>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs A, int64_t rows) {
  constexpr int X = D / 4, R = 256 / (X * Y);   // rows of a workgroup
  __shared__ float4_t part[256 / X][X];
  __shared__ float part_l[256 / X];
  const int x = threadIdx.x % X, z = threadIdx.x / X, y = z % Y, n = A.splits;
  const int64_t row = min((int64_t)blockIdx.x * R + z / Y, rows - 1);
  const int first = unwritten(A.b.cu), end = unwritten(A.b.cu + A.b.seqs);
  const float2* ml = A.ws_ml + row * n;
  const float4_t* src = reinterpret_cast<const float4_t*>(A.ws_o) + row * n * X + x;
  float top = kNoMax;
  for (int i = x; i < n; i += X) top = fmaxf(top, ml[i].x);
#pragma unroll
  for (int d = X / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  float4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  float total = 0.0f;
#pragma unroll 4
  for (int i = y; i < n; i += Y) {
    const float2 v = ml[i];
    const float f = __builtin_amdgcn_exp2f(v.x - top);
    total += v.y * f;
    acc += src[(int64_t)i * X] * f;
  }
  if (Y > 1) {
    part[z][x] = acc;
    if (x == 0) part_l[z] = total;
    __syncthreads();
    if (y != 0) return;
    total = 0.0f;
    acc = (float4_t){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < Y; ++i) {
      total += part_l[z + i];
      acc += part[z + i][x];
    }
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t tok = row / A.hq, hh = row % A.hq;
  if (tok < first || tok >= end) return;
  store4(reinterpret_cast<uint16_t*>(A.out.p + tok * A.out.stride + hh * D + 4 * x), acc * inv, 4, true);
}

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A workgroup of the join has D / 4 threads a row: it takes 8 or 16 rows of up to kFewSplits splits, or one of more.
constexpr int join_rows(int dim) { return 256 / (dim / 4); }
constexpr int kFewSplits = 4;

template <int D, int FMT>
hipError_t go(const AttnArgs& A, const AttnPlan& p, hipStream_t s) {
  const dim3 g((unsigned)p.groups), ts(64 * kWaves), t(256);
  hipError_t e = hipSuccess;
  if (p.nt == 0) {
    e = launch_attn_rows(A, D, FMT, p, s);
    if (p.slices) return e;
  } else {
    if (p.nt == 1) k_attn_split<D, FMT, 1><<<g, ts, 0, s>>>(A);
    if (p.nt == 2) k_attn_split<D, FMT, 2><<<g, ts, 0, s>>>(A);
    if constexpr (D == 64) {
      if (p.nt == 4) k_attn_split<D, FMT, 4><<<g, ts, 0, s>>>(A);
    }
    e = hipGetLastError();
  }
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t rows = (int64_t)A.b.tokens * A.hq;
  const dim3 j((unsigned)p.joins);
  if (p.splits <= kFewSplits)
    k_attn_join<D, 1><<<j, t, 0, s>>>(A, rows);
  else
    k_attn_join<D, join_rows(D)><<<j, t, 0, s>>>(A, rows);
  return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(int hk, int hq, int dim, int64_t seqs, int64_t tokens, int64_t max_new, int64_t max_len) {
  AttnPlan p{};
  if (max_new > tokens && tokens > 0) max_new = tokens;
  const int64_t rows = max_new * (hq / hk), blocks = up(max_len, kKvBlock);
  int64_t one, splits;
  // Up to 32 rows of 128 elements (64 of 64) run on the kernel for few rows, whatever their number of blocks; beyond
  // that it was slower: 64 rows of 128 took 32.8 us against 26.9 (8 sequences of 3000 tokens), 60 rows of 60 tokens 16.8
  // against 7.5; 64 rows of 64 elements 18.5 against 24.3.
  if (rows <= (dim == 64 ? 64 : 32)) {
    p.nt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    // split the cache until every CU has a workgroup, but leave a wave two blocks: 512 and 1024 workgroups read 2 to 20 %
    // slower (1 x 30000, 2 x 65500, 4 x 8000 tokens), with fewer blocks a wave to overlap and more to join
    p.row_tiles = (int)up(rows, 16 * p.nt);
    one = seqs * p.row_tiles * hk;
    splits = one > 0 ? std::min(up(256, one), up(blocks, 2 * kWaves)) : 1;
  } else {
    // Row tiles that there are, as far as the host can tell: the tokens give their number where sequences differ in
    // length. While they leave half of the places on the GPU idle the cache is split to fill them once, in parts of 4
    // blocks at least. While they do not fill the places twice they run in slices of one size (kv_attn_rows.hip): 3
    // prompts of 500 to 2000 on up to 4000 188 us, in splits 204 to 312 for one to four of them; few tiles the other way: 16
    // tokens on 3000 29 us in slices, 13 in splits. Else one workgroup a tile.
    const int64_t tile = attn_rows(dim), places = 256 * 256 / tile;
    p.row_tiles = (int)up(rows, tile);
    one = seqs * p.row_tiles * hk;
    const int64_t there = std::min(seqs * p.row_tiles, tokens * (hq / hk) / tile + seqs) * hk;
    p.slices = one > 0 && blocks >= 16 && 2 * there > places && there < 2 * places;
    splits = one > 0 && blocks >= 16 && 2 * there <= places ? std::min(places / there, up(blocks, 4)) : 1;
  }
  if (splits > 256) splits = 256;
  p.chunk = (int)up(blocks, splits);
  p.splits = (int)up(blocks, p.chunk);
  p.groups = one * p.splits;
  p.threads = p.nt > 0 ? 64 * kWaves : 2 * attn_rows(dim);
  if (p.slices) {
    p.groups = 256 * 256 / attn_rows(dim);
    p.bytes = (size_t)p.groups * (2 * attn_rows(dim) * ((size_t)dim * 4 + 8) + sizeof(SlicePart));
    return p;
  }
  if (p.splits > 1) p.joins = p.splits <= kFewSplits ? up(tokens * hq, join_rows(dim)) : tokens * hq;
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
  const size_t parts = plan.slices ? (size_t)plan.groups * 2 * attn_rows(dim) : (size_t)b.tokens * hq * plan.splits;
  A.ws_ml = reinterpret_cast<float2*>(A.ws_o + parts * dim);
  A.ws_parts = reinterpret_cast<SlicePart*>(A.ws_ml + parts);
  if (dim == 64)
    return format == MQ_KV_INT8 ? go<64, MQ_KV_INT8>(A, plan, s) : go<64, MQ_KV_E4M3>(A, plan, s);
  return format == MQ_KV_INT8 ? go<128, MQ_KV_INT8>(A, plan, s) : go<128, MQ_KV_E4M3>(A, plan, s);
}

}  // namespace mq
