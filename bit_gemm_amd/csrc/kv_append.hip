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
//   open block   the tokens of the block that stays open go into the tail; by
//                the workgroup of the first touched block where that reads the
//                tail, after its reads, since they may take the same places.
// Bound by HBM for prompts (rows read once, codes written once), by the chain
// of dependent loads (offsets, position, rotation, store) for single tokens.
// 4 prompts of 700 to 4096 tokens, 32 query and 8 kv heads of 128 (185 MB): 37 us
// where a large copy would take 36; one token of 16 sequences: 6.6 us.
#include <type_traits>

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

// A block's keys and values in LDS: keys as rows (padded by 16 bytes); values transposed, the tokens of an element as
// pairs, swizzled by groups of four pairs so that neither writes along the elements nor reads along the tokens pile up
// on a bank.
template <int D>
struct Tile {
  _Float16 k[kKvBlock][D + 8];
  uint32_t v[D][kKvBlock / 2];
  uint32_t top[4][2];   // largest magnitudes of the waves' keys and values
  uint8_t bad_tok[kKvBlock];
};
__device__ __forceinline__ int pair_place(int d, int pair) { return pair ^ (((d >> 3) & 7) << 2); }

template <int D>
__device__ __forceinline__ void put_value(Tile<D>& t, int tok, int d, _Float16 x) {
  reinterpret_cast<_Float16*>(&t.v[d][pair_place(d, tok >> 1)])[tok & 1] = x;
}

// The 64 keys and values of the block at p0 of sequence q into LDS, the new keys turned. VEC: the rotation, if any,
// works on whole pieces of 8 elements.
template <int D, bool VEC>
__device__ __forceinline__ void stage(Tile<D>& t, const KvView& kv, const Seq& q, int h, int p0, RowsIn kr, RowsIn vr,
                                      const RopeView& rope) {
  const int tid = threadIdx.x, before = q.len - q.n;   // tokens that were there
  const int have = min(max(before - p0, 0), kKvBlock);
  const _Float16* kx = kr.p + (int64_t)(q.q0 + p0 - before) * kr.stride + (int64_t)h * D;   // token 0's row, new or not
  const _Float16* vx = vr.p + (int64_t)(q.q0 + p0 - before) * vr.stride + (int64_t)h * D;
  // the block's earlier tokens, turned when they came: requested first, laid last
  constexpr int TP = kKvBlock * (D / 8) / 256;
  half8_t kt[TP], vt[TP];
  if (have > 0) {
    const int64_t base = ((int64_t)max(q.slot, 0) * kv.hk + h) * kKvBlock * D;
#pragma unroll
    for (int i = 0; i < TP; ++i) {   // the whole tail: what is not the sequence's is not looked at
      kt[i] = *reinterpret_cast<const half8_t*>(kv.kt + base + 8 * (tid + 256 * i));
      vt[i] = *reinterpret_cast<const half8_t*>(kv.vt + base + 8 * (tid + 256 * i));
    }
  }
  if (VEC) {
    // values: the same piece of two tokens, so that a pair is written whole (half of it may be an older token's, below)
    constexpr int VP = kKvBlock / 2 * (D / 8) / 256;
    half8_t va[VP], vb[VP];
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int e = tid + 256 * i, pair = e / (D / 8), d = 8 * (e % (D / 8));
      va[i] = vb[i] = (half8_t)(_Float16)0.0f;
      if (2 * pair >= have) va[i] = load8(vx + (int64_t)(2 * pair) * vr.stride + d);
      if (2 * pair + 1 >= have) vb[i] = load8(vx + (int64_t)(2 * pair + 1) * vr.stride + d);
    }
    const int half = rope.rot >> 1, turns = !rope.table ? 0 : rope.interleaved ? rope.rot >> 3 : rope.rot >> 4;
    const int rest = rope.table ? (D - rope.rot) >> 3 : D / 8, units = turns + rest;
    const auto key_piece = [&](int tok, int d) {
      return load8(kx + (int64_t)tok * kr.stride + d);
    };
    for (int e = tid; e < kKvBlock * units; e += 256) {
      const int tok = e / units, u = e % units;
      if (tok < have) continue;
      if (u >= turns) {
        const int d = (rope.table ? rope.rot : 0) + 8 * (u - turns);
        *reinterpret_cast<half8_t*>(&t.k[tok][d]) = key_piece(tok, d);
      } else if (rope.interleaved) {
        half8_t a = key_piece(tok, 8 * u);
        float2 cs[4];
        load_cos_sin<4>(rope, p0 + tok, 4 * u, 1.0f, cs);
        turn_piece<true, 4>(a, a, cs);
        *reinterpret_cast<half8_t*>(&t.k[tok][8 * u]) = a;
      } else {
        half8_t a = key_piece(tok, 8 * u), b = key_piece(tok, 8 * u + half);
        float2 cs[8];
        load_cos_sin<8>(rope, p0 + tok, 8 * u, 1.0f, cs);
        turn_piece<false, 8>(a, b, cs);
        *reinterpret_cast<half8_t*>(&t.k[tok][8 * u]) = a;
        *reinterpret_cast<half8_t*>(&t.k[tok][8 * u + half]) = b;
      }
    }
#pragma unroll
    for (int i = 0; i < VP; ++i) {
      const int e = tid + 256 * i, pair = e / (D / 8), d = 8 * (e % (D / 8));
#pragma unroll
      for (int x = 0; x < 8; ++x)
        t.v[d + x][pair_place(d, pair)] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)va[i][x]) |
                                          (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)vb[i][x]) << 16;
    }
    if (have > 0) __syncthreads();   // the older tokens' halves of pairs come after
  } else {
    for (int e = tid; e < kKvBlock * D; e += 256) {
      const int tok = e / D, d = e % D;
      if (tok < have) continue;
      const _Float16* x = kx + (int64_t)tok * kr.stride;
      t.k[tok][d] = rope.table ? turned(x, d, rope, p0 + tok) : x[d];
      put_value(t, tok, d, vx[(int64_t)tok * vr.stride + d]);
    }
  }
  if (have > 0) {
#pragma unroll
    for (int i = 0; i < TP; ++i) {
      const int e = tid + 256 * i, tok = e / (D / 8), d = e >> 3, vtok = 8 * (e & 7);
      if (tok < have) *reinterpret_cast<half8_t*>(&t.k[tok][8 * (e % (D / 8))]) = kt[i];
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (vtok + x < have) put_value(t, vtok + x, d, vt[i][x]);
    }
  }
}

// Largest magnitude of 16 fp16 values, as its bits: the order of the bits is that of the magnitudes, and what is not
// finite lies above all that is.
__device__ __forceinline__ uint32_t top_bits(const half8_t& a, const half8_t& b, uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = __builtin_bit_cast(uint16_t, (_Float16)a[i]) & 0x7FFFu;
    const uint32_t y = __builtin_bit_cast(uint16_t, (_Float16)b[i]) & 0x7FFFu;
    top = max(top, max(x, y));
  }
  return top;
}

template <int FMT>
__device__ __forceinline__ uint4 code16(const half8_t& a, const half8_t& b, float inv) {
  uint4 w;
  w.x = code4<FMT>((float)a[0] * inv, (float)a[1] * inv, (float)a[2] * inv, (float)a[3] * inv);
  w.y = code4<FMT>((float)a[4] * inv, (float)a[5] * inv, (float)a[6] * inv, (float)a[7] * inv);
  w.z = code4<FMT>((float)b[0] * inv, (float)b[1] * inv, (float)b[2] * inv, (float)b[3] * inv);
  w.w = code4<FMT>((float)b[4] * inv, (float)b[5] * inv, (float)b[6] * inv, (float)b[7] * inv);
  return w;
}

// Scales and codes of the block in LDS into block `id` of head h: a thread codes pieces of 16 elements of the keys' rows
// and of the values' columns, contiguous in memory over the lanes.
template <int D, int FMT>
__device__ __forceinline__ void code_block(Tile<D>& t, const KvView& kv, int64_t id, int h) {
  constexpr float kMax = FMT == MQ_KV_INT8 ? 127.0f : 448.0f;
  constexpr int P = kKvBlock * D / 16 / 256;   // pieces of a thread
  const int tid = threadIdx.x;
  half8_t k[P][2], v[P][2];
  uint32_t kt = 0, vt = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int p = tid + 256 * i, tok = p / (D / 16), kd = 16 * (p % (D / 16)), d = p / 4, pair = 8 * (p % 4);
    k[i][0] = *reinterpret_cast<const half8_t*>(&t.k[tok][kd]);
    k[i][1] = *reinterpret_cast<const half8_t*>(&t.k[tok][kd + 8]);
    v[i][0] = *reinterpret_cast<const half8_t*>(&t.v[d][pair_place(d, pair)]);
    v[i][1] = *reinterpret_cast<const half8_t*>(&t.v[d][pair_place(d, pair + 4)]);
    kt = top_bits(k[i][0], k[i][1], kt);
    vt = top_bits(v[i][0], v[i][1], vt);
  }
  const auto join = [&]() {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      kt = max(kt, (uint32_t)__shfl_xor((int)kt, d));
      vt = max(vt, (uint32_t)__shfl_xor((int)vt, d));
    }
    if ((tid & 63) == 0) {
      t.top[tid >> 6][0] = kt;
      t.top[tid >> 6][1] = vt;
    }
    __syncthreads();
    kt = max(max(t.top[0][0], t.top[1][0]), max(t.top[2][0], t.top[3][0]));
    vt = max(max(t.top[0][1], t.top[1][1]), max(t.top[2][1], t.top[3][1]));
  };
  join();
  const bool bad = kt >= 0x7C00u || vt >= 0x7C00u;
  if (bad) {
    // rare: vectors that are not finite. Their key rows count as zeros, and so do the values that are no numbers.
    if (tid < kKvBlock) t.bad_tok[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int p = tid + 256 * i, tok = p / (D / 16), vtok = 16 * (p % 4);
      if (top_bits(k[i][0], k[i][1], 0) >= 0x7C00u) t.bad_tok[tok] = 1;
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        if (!finite_h(v[i][x >> 3][x & 7])) {
          t.bad_tok[vtok + x] = 1;
          v[i][x >> 3][x & 7] = (_Float16)0.0f;
        }
      }
    }
    __syncthreads();
    kt = vt = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (t.bad_tok[(tid + 256 * i) / (D / 16)]) k[i][0] = k[i][1] = (half8_t)(_Float16)0.0f;
      kt = top_bits(k[i][0], k[i][1], kt);
      vt = top_bits(v[i][0], v[i][1], vt);
    }
    join();
  }
  const float km = h_to_f(kt), vm = h_to_f(vt);
  const float ki = km > 0.0f ? kMax * (1.0f / km) : 0.0f, vi = vm > 0.0f ? kMax * (1.0f / vm) : 0.0f;
  const int64_t head = id * kv.hk + h;
  uint4* ko = reinterpret_cast<uint4*>(kv.kc + head * (kKvBlock * D));
  uint4* vo = reinterpret_cast<uint4*>(kv.vc + head * (kKvBlock * D));
#pragma unroll
  for (int i = 0; i < P; ++i) {
    ko[tid + 256 * i] = code16<FMT>(k[i][0], k[i][1], ki);
    vo[tid + 256 * i] = code16<FMT>(v[i][0], v[i][1], vi);
  }
  if (tid == 0) {
    // the keys carry the mark of a vector that is not finite: a NaN scale makes the head's scores NaN for the rows that
    // attend to the block, and masked scores are replaced before use
    kv.ks[head] = bad ? __builtin_nanf("") : km / kMax;
    kv.vs[head] = vm / kMax;
  }
}

// Queries of one sequence: tokens t0 .. t1 - 1 turned.
template <int D, bool VEC>
__device__ __forceinline__ void turn_queries(const Seq& q, int t0, int t1, int hq, RowsIn qr, RowsOut qo,
                                             const RopeView& rope) {
  const int64_t pos0 = (int64_t)q.len - q.n;
  if (VEC) {
    constexpr int HP = 4;   // heads that share the cosines and sines a thread loads
    const int half = rope.rot >> 1, turns = rope.interleaved ? rope.rot >> 3 : rope.rot >> 4;
    const int units = turns + ((D - rope.rot) >> 3), hg = (hq + HP - 1) / HP, per = hg * units;
    for (int e = threadIdx.x; e < (t1 - t0) * per; e += 256) {
      const int tok = t0 + e / per, rest = e % per, h0 = rest / units * HP, u = rest % units;
      const _Float16* x = qr.p + (int64_t)(q.q0 + tok) * qr.stride + (int64_t)h0 * D;
      _Float16* y = qo.p + (int64_t)(q.q0 + tok) * qo.stride + (int64_t)h0 * D;
      const bool pass = u >= turns;
      const int d = pass ? rope.rot + 8 * (u - turns) : 8 * u;
      const bool two = !pass && !rope.interleaved;
      half8_t a[HP], b[HP];
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        if (h0 + h < hq) {
          a[h] = load8(x + h * D + d);
          if (two) b[h] = load8(x + h * D + d + half);
        }
      }
      float2 cs[8];
      if (two)
        load_cos_sin<8>(rope, pos0 + tok, 8 * u, 1.0f, cs);
      else if (!pass)
        load_cos_sin<4>(rope, pos0 + tok, 4 * u, 1.0f, cs);
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        if (h0 + h < hq) {
          if (two) {
            turn_piece<false, 8>(a[h], b[h], cs);
            store8(y + h * D + d + half, b[h]);
          } else if (!pass) {
            turn_piece<true, 4>(a[h], a[h], cs);
          }
          store8(y + h * D + d, a[h]);
        }
      }
    }
  } else {
    const int pairs = rope.rot >> 1, units = pairs + D - rope.rot, per = hq * units;
    for (int e = threadIdx.x; e < (t1 - t0) * per; e += 256) {
      const int tok = t0 + e / per, rest = e % per, h = rest / units, u = rest % units;
      const _Float16* x = qr.p + (int64_t)(q.q0 + tok) * qr.stride + (int64_t)h * D;
      _Float16* y = qo.p + (int64_t)(q.q0 + tok) * qo.stride + (int64_t)h * D;
      if (u >= pairs) {
        y[rope.rot + u - pairs] = x[rope.rot + u - pairs];
      } else {
        const int i0 = rope.interleaved ? 2 * u : u, i1 = rope.interleaved ? i0 + 1 : u + pairs;
        const float2 r = turn((float)x[i0], (float)x[i1], cos_sin(rope, pos0 + tok, u));
        y[i0] = (_Float16)r.x;
        y[i1] = (_Float16)r.y;
      }
    }
  }
}

template <int D, int FMT, bool VEC>
__global__ __launch_bounds__(256) void k_append(KvView kv, BatchView b, RowsIn qr, int hq, RowsIn kr, RowsIn vr,
                                                RopeView rope, RowsOut qo, int touched, int kv_groups,
                                                int q_tokens, int q_groups) {
  const int tid = threadIdx.x;
  if ((int)blockIdx.x >= kv_groups) {
    const int w = (int)blockIdx.x - kv_groups;
    const int s = w / q_groups, t0 = (w % q_groups) * q_tokens;
    const Seq q = seq_of(b, kv, s);
    turn_queries<D, VEC>(q, t0, min(q.n, t0 + q_tokens), hq, qr, qo, rope);
    return;
  }
  __shared__ __attribute__((aligned(16))) Tile<D> tile;
  const int h = (int)blockIdx.x % kv.hk, rest = (int)blockIdx.x / kv.hk, j = rest % touched, s = rest / touched;
  const Seq q = seq_of(b, kv, s);
  if (q.n == 0) return;
  const int before = q.len - q.n;
  const int first = max(before, 0) / kKvBlock, last_full = q.cap / kKvBlock;   // blocks before last_full are full
  const int blk = first + j;
  if (blk < last_full) {
    const int p0 = blk * kKvBlock;
    const int id = b.table[(int64_t)s * b.width + blk];
    // a block that cannot be written is dropped; so is one whose earlier tokens have no slot to come from
    if ((uint64_t)(int64_t)id < (uint64_t)kv.blocks && (before <= p0 || q.slot >= 0)) {
      stage<D, VEC>(tile, kv, q, h, p0, kr, vr, rope);
      __syncthreads();
      code_block<D, FMT>(tile, kv, id, h);
    }
  }
  // The tokens that stay open: by the workgroup of their block, but after the first block's reads of the tail where it
  // has any and becomes full, since they may take the same places.
  const int open0 = last_full * kKvBlock, from = max(max(before, 0), open0);
  const int owner = before > first * kKvBlock && first < last_full ? 0 : last_full - first;
  if (j != owner || q.slot < 0 || from >= q.cap) return;
  __syncthreads();
  const int wave = tid >> 6, lane = tid & 63;
  const int64_t base = ((int64_t)q.slot * kv.hk + h) * kKvBlock * D;
  constexpr int E = D / 64, B = 4;   // elements of a lane, tokens a wave has under way at once
  for (int p0 = from + wave; p0 < q.cap; p0 += 4 * B) {
    _Float16 a[B][E], v[B][E];
#pragma unroll
    for (int t = 0; t < B; ++t) {
      const int p = min(p0 + 4 * t, q.cap - 1);
      const int64_t row = q.q0 + p - before;
      const _Float16* xk = kr.p + row * kr.stride + (int64_t)h * D;
      const _Float16* xv = vr.p + row * vr.stride + (int64_t)h * D;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int d = lane + 64 * i;
        a[t][i] = rope.table ? turned(xk, d, rope, p) : xk[d];
        v[t][i] = xv[d];
      }
    }
#pragma unroll
    for (int t = 0; t < B; ++t) {
      const int p = p0 + 4 * t;
      if (p >= q.cap) break;
      bool bad = false;
#pragma unroll
      for (int i = 0; i < E; ++i) bad |= !finite_h(a[t][i]) || !finite_h(v[t][i]);
      // a vector that is not finite: the key row is NaN as a whole (its scores are NaN, and only its),
      // the value column holds zeros in its place, so that a masked token multiplies nothing but numbers
      const bool any = __any(bad);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int d = lane + 64 * i;
        kv.kt[base + (int64_t)(p - open0) * D + d] = any ? (_Float16)__builtin_nanf("") : a[t][i];
        kv.vt[base + (int64_t)d * kKvBlock + (p - open0)] = finite_h(v[t][i]) ? v[t][i] : (_Float16)0.0f;
      }
    }
  }
}

template <int D, int FMT>
hipError_t go(const KvView& kv, const BatchView& b, RowsIn q, int hq, RowsIn k, RowsIn v, const RopeView& rope,
              RowsOut qo, int touched, int kv_groups, int q_tokens, int q_groups, int groups, hipStream_t s) {
  const dim3 g((unsigned)groups), t(256);
  const bool vec = !rope.table || piecewise(rope);
  if (vec)
    k_append<D, FMT, true><<<g, t, 0, s>>>(kv, b, q, hq, k, v, rope, qo, touched, kv_groups, q_tokens, q_groups);
  else
    k_append<D, FMT, false><<<g, t, 0, s>>>(kv, b, q, hq, k, v, rope, qo, touched, kv_groups, q_tokens, q_groups);
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
  if (!launchable(groups, 256)) {
    *grid_too_large = true;
    return hipSuccess;
  }
  const auto run = [&](auto d, auto f) {
    return go<decltype(d)::value, decltype(f)::value>(kv, b, q, hq, k, v, rope, qo, (int)touched, (int)kv_groups,
                                                      (int)q_tokens, (int)q_groups, (int)groups, s);
  };
  using std::integral_constant;
  if (dim == 64)
    return format == MQ_KV_INT8 ? run(integral_constant<int, 64>{}, integral_constant<int, MQ_KV_INT8>{})
                                : run(integral_constant<int, 64>{}, integral_constant<int, MQ_KV_E4M3>{});
  return format == MQ_KV_INT8 ? run(integral_constant<int, 128>{}, integral_constant<int, MQ_KV_INT8>{})
                              : run(integral_constant<int, 128>{}, integral_constant<int, MQ_KV_E4M3>{});
}

}  // namespace mq
