// The append to the 8-bit key/value cache (include/mosaicq_block.h,
// mq_kv_append), with the rotation of queries and keys in the same launch.
//
// One launch, three kinds of workgroups of 256 threads:
//   queries      some tokens of one sequence: read, turned, written;
//   full blocks  one (sequence, block that the new tokens touch, kv head): 64
//                tokens of keys and values come from the new rows (keys turned)
//                or, for the block's earlier tokens, from the tail; the largest
//                magnitude of each gives its scale; codes are written, the
//                values' transposed, so that the attention reads both as the
//                matrix cores want them without a transposition of its own;
//   open block   the workgroup of a sequence's first touched block also writes
//                the tokens of the block that stays open into the tail: after
//                its own reads of the tail, which may share the tail's places.
// Bound by HBM for prompts (rows read once, codes written once), by the chain
// of dependent loads (offsets, position, rotation, store) for single tokens.
#include "block_common.h"

namespace mq {
namespace {

template <int FMT>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
  if (FMT == MQ_KV_INT8) {
    const auto one = [](float v) { return (uint32_t)(int)rintf(fminf(fmaxf(v, -127.0f), 127.0f)) & 255u; };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
  const auto cut = [](float v) { return fminf(fmaxf(v, -448.0f), 448.0f); };
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cut(a), cut(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cut(c), cut(d), (int)w, true);
}

template <int D>
struct Tile {
  _Float16 x[kKvBlock][D + 8];   // rows padded by 16 bytes: column reads spread over the banks
};

// The 64 keys or values of block `blk` of sequence q into LDS, turned.
template <int D, bool IS_K>
__device__ __forceinline__ void stage(Tile<D>& t, const KvView& kv, const Seq& q, int h, int p0, RowsIn rows,
                                      const RopeView& rope) {
  const int before = q.len - q.n;   // tokens that were there
  const int have = min(max(before - p0, 0), kKvBlock);
  if (have > 0) {
    const int64_t base = ((int64_t)max(q.slot, 0) * kv.hk + h) * kKvBlock * D;
    for (int e = threadIdx.x; e < kKvBlock * D; e += 256) {
      const int tok = IS_K ? e / D : e % kKvBlock, d = IS_K ? e % D : e / kKvBlock;
      if (tok < have) t.x[tok][d] = (IS_K ? kv.kt : kv.vt)[base + e];
    }
  }
  for (int e = threadIdx.x; e < kKvBlock * D; e += 256) {
    const int tok = e / D, d = e % D;
    if (tok >= have) {
      const _Float16* x = rows.p + (int64_t)(q.q0 + p0 + tok - before) * rows.stride + (int64_t)h * D;
      t.x[tok][d] = IS_K && rope.table ? turned(x, d, rope, p0 + tok) : x[d];
    }
  }
}

template <int D, int FMT>
__global__ __launch_bounds__(256) void k_append(KvView kv, BatchView b, RowsIn qr, int hq, RowsIn kr, RowsIn vr,
                                                RopeView rope, RowsOut qo, int touched, int kv_groups,
                                                int q_tokens, int q_groups) {
  constexpr float kMax = FMT == MQ_KV_INT8 ? 127.0f : 448.0f;
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= kv_groups) {   // queries
    const int w = (int)blockIdx.x - kv_groups;
    const int s = w / q_groups, t0 = (w % q_groups) * q_tokens;
    const Seq q = seq_of(b, kv, s);
    const int t1 = min(q.n, t0 + q_tokens);
    const int pairs = rope.rot >> 1, units = pairs + D - rope.rot, per = hq * units;
    for (int e = tid; e < (t1 - t0) * per; e += 256) {
      const int tok = t0 + e / per, rest = e % per, h = rest / units, u = rest % units;
      const _Float16* x = qr.p + (int64_t)(q.q0 + tok) * qr.stride + (int64_t)h * D;
      _Float16* y = qo.p + (int64_t)(q.q0 + tok) * qo.stride + (int64_t)h * D;
      if (u >= pairs) {
        y[rope.rot + u - pairs] = x[rope.rot + u - pairs];
      } else {
        const int i0 = rope.interleaved ? 2 * u : u, i1 = rope.interleaved ? i0 + 1 : u + pairs;
        const float2 r = turn((float)x[i0], (float)x[i1], cos_sin(rope, (int64_t)q.len - q.n + tok, u));
        y[i0] = (_Float16)r.x;
        y[i1] = (_Float16)r.y;
      }
    }
    return;
  }
  __shared__ Tile<D> lk, lv;
  __shared__ float red[4][2];
  __shared__ int bad_any;
  __shared__ uint8_t bad_tok[kKvBlock];
  const int h = (int)blockIdx.x % kv.hk, rest = (int)blockIdx.x / kv.hk, j = rest % touched, s = rest / touched;
  const Seq q = seq_of(b, kv, s);
  const int before = q.len - q.n;
  const int first = max(before, 0) / kKvBlock, last_full = q.cap / kKvBlock;   // blocks before last_full are full
  if (q.n == 0) return;
  const int blk = first + j;
  if (blk < last_full) {
    const int p0 = blk * kKvBlock;
    const int id = b.table[(int64_t)s * b.width + blk];
    const bool reads_tail = before > p0;
    // a block that cannot be written is dropped; so is one whose earlier tokens have no slot to come from
    const bool ok = (uint64_t)(int64_t)id < (uint64_t)kv.blocks && (!reads_tail || q.slot >= 0);
    if (ok) {
      if (tid == 0) bad_any = 0;
      if (tid < kKvBlock) bad_tok[tid] = 0;
      stage<D, true>(lk, kv, q, h, p0, kr, rope);
      stage<D, false>(lv, kv, q, h, p0, vr, rope);
      __syncthreads();
      // a quarter of a key row each, the values by columns: D / 4 elements of both a thread
      constexpr int E = D / 4;
      const int kt = tid >> 2, kd = (tid & 3) * E;
      const int vd = tid / (256 / D), vt = (tid % (256 / D)) * E;   // 64 tokens / (256 / D) = D / 4
      float ka[E], va[E], km = 0.0f, vm = 0.0f;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const _Float16 x = lk.x[kt][kd + i], y = lv.x[vt + i][vd];
        const bool fx = finite_h(x), fy = finite_h(y);
        bad |= !fx || !fy;
        if (!fx) bad_tok[kt] = 1;
        if (!fy) bad_tok[vt + i] = 1;
        ka[i] = fx ? (float)x : 0.0f;
        va[i] = fy ? (float)y : 0.0f;
        km = fmaxf(km, fabsf(ka[i]));
        vm = fmaxf(vm, fabsf(va[i]));
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        km = fmaxf(km, __shfl_xor(km, d));
        vm = fmaxf(vm, __shfl_xor(vm, d));
      }
      if ((tid & 63) == 0) {
        red[tid >> 6][0] = km;
        red[tid >> 6][1] = vm;
      }
      if (bad) bad_any = 1;
      __syncthreads();
      km = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
      vm = fmaxf(fmaxf(red[0][1], red[1][1]), fmaxf(red[2][1], red[3][1]));
      if (bad_any) {   // rare: the key rows of vectors that are not finite count as zeros, as they do from the tail
        __syncthreads();
        if (bad_tok[kt]) {
#pragma unroll
          for (int i = 0; i < E; ++i) ka[i] = 0.0f;
        }
        km = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) km = fmaxf(km, fabsf(ka[i]));
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) km = fmaxf(km, __shfl_xor(km, d));
        if ((tid & 63) == 0) red[tid >> 6][0] = km;
        __syncthreads();
        km = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
      }
      const float ki = km > 0.0f ? kMax * (1.0f / km) : 0.0f, vi = vm > 0.0f ? kMax * (1.0f / vm) : 0.0f;
      const int64_t base = ((int64_t)id * kv.hk + h) * kKvBlock * D;
      uint32_t* ko = reinterpret_cast<uint32_t*>(kv.kc + base + (int64_t)kt * D + kd);
      uint32_t* vo = reinterpret_cast<uint32_t*>(kv.vc + base + (int64_t)vd * kKvBlock + vt);
#pragma unroll
      for (int i = 0; i < E; i += 4) {
        ko[i / 4] = code4<FMT>(ka[i] * ki, ka[i + 1] * ki, ka[i + 2] * ki, ka[i + 3] * ki);
        vo[i / 4] = code4<FMT>(va[i] * vi, va[i + 1] * vi, va[i + 2] * vi, va[i + 3] * vi);
      }
      if (tid == 0) {
        // the keys carry the mark of a vector that is not finite: a NaN scale makes the head's
        // scores NaN for the rows that attend to the block, and masked scores are replaced before use
        kv.ks[(int64_t)id * kv.hk + h] = bad_any ? __builtin_nanf("") : km / kMax;
        kv.vs[(int64_t)id * kv.hk + h] = vm / kMax;
      }
    }
  }
  // the tokens that stay open
  if (j != 0 || q.slot < 0) return;
  const int open0 = last_full * kKvBlock, from = max(max(before, 0), open0);
  if (from >= q.cap) return;
  __syncthreads();   // the tail's tokens of the first block are in registers or written by now
  const int wave = tid >> 6, lane = tid & 63;
  const int64_t base = ((int64_t)q.slot * kv.hk + h) * kKvBlock * D;
  for (int p = from + wave; p < q.cap; p += 4) {
    const int64_t row = q.q0 + p - before;
    const _Float16* xk = kr.p + row * kr.stride + (int64_t)h * D;
    const _Float16* xv = vr.p + row * vr.stride + (int64_t)h * D;
    _Float16 a[D / 64], v[D / 64];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int d = lane + 64 * i;
      a[i] = rope.table ? turned(xk, d, rope, p) : xk[d];
      v[i] = xv[d];
      bad |= !finite_h(a[i]) || !finite_h(v[i]);
    }
    // a vector that is not finite: the key row is NaN as a whole (its scores are NaN, and only its),
    // the value column holds zeros in its place, so that a masked token multiplies nothing but numbers
    const bool any = __any(bad);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int d = lane + 64 * i;
      kv.kt[base + (int64_t)(p - open0) * D + d] = any ? (_Float16)__builtin_nanf("") : a[i];
      kv.vt[base + (int64_t)d * kKvBlock + (p - open0)] = finite_h(v[i]) ? v[i] : (_Float16)0.0f;
    }
  }
}

template <int D>
hipError_t go(const KvView& kv, int format, const BatchView& b, RowsIn q, int hq, RowsIn k, RowsIn v,
              const RopeView& rope, RowsOut qo, int touched, int kv_groups, int q_tokens, int q_groups, int groups,
              hipStream_t s) {
  const dim3 g((unsigned)groups), t(256);
  if (format == MQ_KV_INT8)
    k_append<D, MQ_KV_INT8><<<g, t, 0, s>>>(kv, b, q, hq, k, v, rope, qo, touched, kv_groups, q_tokens, q_groups);
  else
    k_append<D, MQ_KV_E4M3><<<g, t, 0, s>>>(kv, b, q, hq, k, v, rope, qo, touched, kv_groups, q_tokens, q_groups);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvView& kv, int dim, int format, const BatchView& b, RowsIn q, int hq, RowsIn k,
                            RowsIn v, const RopeView& rope, RowsOut qo, bool* grid_too_large, hipStream_t s) {
  *grid_too_large = false;
  if (b.seqs == 0 || b.tokens == 0) return hipSuccess;
  const int64_t new_max = b.max_new < b.tokens ? b.max_new : b.tokens;
  // new tokens that start on a block's last place touch the most blocks
  const int64_t touched = (new_max + 2 * kKvBlock - 2) / kKvBlock;
  const int64_t kv_groups = (int64_t)b.seqs * touched * kv.hk;
  const int64_t q_tokens = 4;
  const int64_t q_groups = rope.table && q.p ? (new_max + q_tokens - 1) / q_tokens : 0;
  const int64_t groups = kv_groups + q_groups * b.seqs;
  if (groups >= (int64_t(1) << 31)) {
    *grid_too_large = true;
    return hipSuccess;
  }
  return dim == 64 ? go<64>(kv, format, b, q, hq, k, v, rope, qo, (int)touched, (int)kv_groups, (int)q_tokens,
                            (int)q_groups, (int)groups, s)
                   : go<128>(kv, format, b, q, hq, k, v, rope, qo, (int)touched, (int)kv_groups, (int)q_tokens,
                             (int)q_groups, (int)groups, s);
}

}  // namespace mq
