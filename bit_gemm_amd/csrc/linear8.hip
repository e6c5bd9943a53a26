// The product of 8-bit rows with 8-bit weights (include/mosaicq_head.h,
// mq_linear8):
//
//   Y[m][n] = sum over blocks b of 128 of 2^(ex[m][b] + ew[n][b]) sum_k x[m][k] w[n][k]
//
// on the fp8 matrix instruction of 128 columns, which takes both scales as
// exponent bytes and applies them itself. The weights are the A operand, so a
// lane holds four outputs of a token that follow each other.
#include <utility>

#include "head_internal.h"
#include "kernel_common.h"
#include "q8.h"

namespace mq {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 2048;      // bytes of 16 rows x 128 columns

// D += 2^(sa - 127) A 2^(sb - 127) B: lane l supplies row (A) and column (B) l % 16, the 32 columns 16 (l / 16) + 0..15 and
// 64 + 16 (l / 16) + 0..15 of the block, and byte J of its scale words; it receives D[4 (l / 16) + 0..3][l % 16]. (Which
// columns a lane holds is free, where A and B hold the same and one scale goes for all 128.)
template <int J>
__device__ __forceinline__ float4_t mfma8(i32x8_t a, i32x8_t b, float4_t c, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, J, sa, J, sb);
}

__device__ __forceinline__ i32x8_t join(i32x4_t a, i32x4_t b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

__device__ __forceinline__ i32x8_t load_halves(const uint8_t* p, int apart) {
  return join(*reinterpret_cast<const i32x4_t*>(p), *reinterpret_cast<const i32x4_t*>(p + apart));
}

// The scale bytes of blocks 4 q .. 4 q + 3 of a row of Kt (127 past it), from any address.
typedef uint32_t u32_any_t __attribute__((aligned(1)));
__device__ __forceinline__ int row_scales(const uint8_t* row, int q, int Kt) {
  if (4 * q + 4 <= Kt) return (int)*reinterpret_cast<const u32_any_t*>(row + 4 * q);
  uint32_t v = 0x7F7F7F7Fu;
  for (int j = 0; 4 * q + j < Kt; ++j) v = (v & ~(0xFFu << (8 * j))) | ((uint32_t)row[4 * q + j] << (8 * j));
  return (int)v;
}

__device__ __forceinline__ void put4(_Float16* y, float4_t v, int64_t left) {
  typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
  if (left >= 4 && (reinterpret_cast<uintptr_t>(y) & 7) == 0) {
    *reinterpret_cast<half4_t*>(y) = (half4_t){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) y[i] = (_Float16)v[i];
  }
}

template <typename F, int... J>
__device__ __forceinline__ void four(F&& f, std::integer_sequence<int, J...>) {
  (f(std::integral_constant<int, J>{}), ...);
}

// ------------------------------------------------------------ few tokens
// Up to 16 NT tokens: a workgroup takes R blocks of 16 weight rows, its waves
// fours of tiles along K in turn (a lane's scales of four blocks are one word).
// The weights go from memory straight to the registers that the instruction
// reads, once; the tokens' codes come through L2. The waves' sums meet in LDS
// and are added in their order.
template <int NT, int R>
__global__ __launch_bounds__(512) void k_stream8(Rows8 x, int M, W8 w, _Float16* y, int64_t ys) {
  extern __shared__ float4_t red[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int rb0 = blockIdx.x * R;
  const uint8_t *xc[NT], *xs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t m = min(16 * t + r, M - 1);      // tokens past the last one repeat it; their outputs are not stored
    xc[t] = x.codes + m * x.stride + 16 * g;
    xs[t] = x.scales + m * x.sstride;
  }
  float4_t acc[R][NT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};

  for (int q = wave; q < w.Kq; q += waves) {
    int sw[R], sx[NT];
    i32x8_t a[4][R], b[4][NT];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t rb = min(rb0 + i, w.Nb - 1);
      sw[i] = *reinterpret_cast<const int*>(w.scales + 64 * (rb * w.Kq + q) + 4 * r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kt = min(4 * q + j, w.Kt - 1);
        a[j][i] = load_halves(w.codes + kTile * (rb * w.Kt + kt) + 16 * lane, 1024);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      sx[t] = row_scales(xs[t], q, w.Kt);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j][t] = load_halves(xc[t] + kQ8Block * min(4 * q + j, w.Kt - 1), 64);
    }
    four([&](auto j) {
      if (4 * q + j < w.Kt) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[i][t] = mfma8<j>(a[j][i], b[j][t], acc[i][t], sw[i], sx[t]);
      }
    }, std::make_integer_sequence<int, 4>{});
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) red[(wave * R * NT + i * NT + t) * 64 + lane] = acc[i][t];
  __syncthreads();
  for (int o = threadIdx.x; o < R * NT * 64; o += blockDim.x) {
    float4_t v = red[o];
    for (int k = 1; k < waves; ++k) v += red[k * R * NT * 64 + o];
    const int part = o >> 6, l = o & 63;
    const int64_t m = 16 * (part % NT) + (l & 15), n = 16 * (int64_t)(rb0 + part / NT) + 4 * (l >> 4);
    if (m < M && n < w.N) put4(y + m * ys + n, v, w.N - n);
  }
}

template <int NT, int R>
hipError_t go_stream(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, const Linear8Plan& p,
                     hipStream_t s) {
  const size_t lds = (size_t)p.waves * R * NT * 1024;
  k_stream8<NT, R><<<dim3((unsigned)((w.Nb + R - 1) / R)), dim3(64 * p.waves), lds, s>>>(x, (int)M, w, y, ys);
  return hipGetLastError();
}

// ----------------------------------------------------------- many tokens
// A workgroup of 4 waves makes 64 RB weight rows x 128 tokens; a wave its own
// 16 RB rows with all the tokens. The weights lie in the instruction's order,
// so they go from L2 straight to registers; the tokens' codes go to LDS, where
// the waves share them, by direct copies three blocks of 128 columns ahead (two
// workgroups a CU). Steps are taken by fours, which share the words of scales;
// what lies past K in the last four is zero in LDS and adds nothing. Nothing in
// a step is under a condition: a load there would be waited for where the
// branches meet.
constexpr int kTb = 8;           // blocks of 16 tokens a workgroup
constexpr int kStage = kTb * kTile;
constexpr int kTiledLds = 4 * kStage + 2 * (256 + 256) * 4;      // codes; scale words of the tokens and the weight rows

// The codes of 16 tokens x 128 columns in LDS are filled by two copies of 1 KiB, in lane order. Copy u, lane l brings row
// l / 4, chunk 4 u + (l % 4 ^ row / 2 % 4) of its 8 chunks of 16 bytes: quads read runs of 64 bytes, and the 8 lanes that
// LDS serves at once when the operand is read back (rows n .. n + 7, one chunk) find 8 different banks of 16 bytes.
__device__ __forceinline__ uint32_t stage_chunk(int lane) { return (uint32_t)((lane & 3) ^ ((lane >> 3) & 3)); }
__device__ __forceinline__ uint32_t stage_pos(int lane) {
  const int n = lane & 15, g = lane >> 4;
  return 16u * (uint32_t)(4 * n + (g ^ ((n >> 1) & 3)));
}

// A barrier for LDS alone: loads stay on their way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int RB>
__global__ __launch_bounds__(256, 2) void k_tiled8(Rows8 x, int M, W8 w, _Float16* y, int64_t ys, float* part, int NT,
                                                   int T, int per) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int kAhead = RB == 4 ? 1 : 3;      // steps that the weights are asked for ahead: what the registers hold
  constexpr int kSets = kAhead + 1;
  constexpr int kCopies = 2 * (kTb / 4);       // of a wave in a step
  uint32_t* const scale_lds = reinterpret_cast<uint32_t*>(lds + 4 * kStage);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, g = lane >> 4;
  const int tile = xcd_tile(blockIdx.x, T), MT = T / NT;
  const int nt = tile / MT, mt = tile - nt * MT;
  const int rb0 = (nt * 4 + wave) * RB, m0 = 16 * kTb * mt;
  const int kt0 = blockIdx.y * per, kt1 = min(w.Kt, kt0 + per), q1 = (kt1 + 3) >> 2;

  // the workgroup's token rows; reads past them give zero
  const int rows = min(16 * kTb, M - m0);
  const uint32_t range = (uint32_t)rows * (uint32_t)x.stride;
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(x.codes + (int64_t)m0 * x.stride), 0, (int)range, kBufferRaw);
  const uint32_t xl = (uint32_t)(lane >> 2) * (uint32_t)x.stride + 16u * stage_chunk(lane);
  auto copy = [&](int stage, int kt) {
    const uint32_t at = kt < kt1 ? (uint32_t)kt * kQ8Block : 0x40000000u;      // past the split: zero
#pragma unroll
    for (int i = 0; i < kTb / 4; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tb = (kTb / 4) * wave + i;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            xr, (__attribute__((address_space(3))) void*)(lds + stage * kStage + tb * kTile + 1024 * u), 16,
            xl + (uint32_t)(16 * tb) * (uint32_t)x.stride + at + 64 * u, 0, 0, 0);
      }
  };
  // the wave's weight rows: one offset a lane, the tile's in a scalar register (rows past the last block repeat it)
  const int rbw = min(rb0, w.Nb - 1);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(w.codes + (int64_t)kTile * rbw * w.Kt), 0, 0x7FFFFFFF, kBufferRaw);
  const int wl = 16 * lane;
  i32x8_t a[kSets][RB];
  auto weights = [&](int set, int kt) {
    kt = min(kt, w.Kt - 1);
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int at = (min(i, w.Nb - 1 - rbw) * w.Kt + kt) * kTile;
      a[set][i] = join(__builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, wl, at, 0)),
                       __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wr, wl, at + 1024, 0)));
    }
  };
  // The scales of four blocks: a thread asks for those of a token and of a weight row of the workgroup, and puts them into
  // LDS as words two steps later.
  const uint8_t* const xs = x.scales + (int64_t)min(m0 + (tid & 127), M - 1) * x.sstride;
  const uint8_t* const ws = w.scales + 64 * (int64_t)min(nt * 4 * RB + (tid >> 4), w.Nb - 1) * w.Kq + 4 * (tid & 15);
  uint32_t byte[4], word;
  auto ask_scales = [&](int q) {
#pragma unroll
    for (int j = 0; j < 4; ++j) byte[j] = xs[min(4 * q + j, w.Kt - 1)];
    word = *reinterpret_cast<const uint32_t*>(ws + 64 * min(q, w.Kq - 1));
  };
  auto put_scales = [&](int q) {
    uint32_t* const to = scale_lds + (q & 1) * 512;      // tokens come twice: a branch here would part the step
    to[tid] = byte[0] | (byte[1] << 8) | (byte[2] << 16) | (byte[3] << 24);
    to[256 + tid] = word;
  };

  float4_t acc[RB][kTb];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int t = 0; t < kTb; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};

  const int q0 = kt0 >> 2;
  ask_scales(q0);
#pragma unroll
  for (int j = 0; j < 3; ++j) copy(j, kt0 + j);
#pragma unroll
  for (int j = 0; j < kAhead; ++j) weights(j, kt0 + j);
  put_scales(q0);
  wait_loads<0>();
  lds_barrier();
  const uint32_t pos = stage_pos(lane);
  for (int q = q0; q < q1; ++q) {
    const uint32_t* const scale = scale_lds + (q & 1) * 512;
    int sx[kTb], sw[RB];
#pragma unroll
    for (int t = 0; t < kTb; ++t) sx[t] = (int)scale[16 * t + r];
#pragma unroll
    for (int i = 0; i < RB; ++i) sw[i] = (int)scale[256 + 16 * (wave * RB + i) + r];
    ask_scales(q + 1);
    four([&](auto j) {
      const int kt = 4 * q + j;
      copy((j + 3) & 3, kt + 3);
      weights((j + kAhead) % kSets, kt + kAhead);
      __builtin_amdgcn_sched_barrier(0);        // the loads go out first,
      const uint8_t* const cur = lds + j * kStage + pos;
      i32x8_t b[2];
      b[0] = load_halves(cur, 1024);
#pragma unroll
      for (int t = 0; t < kTb; ++t) {
        if (t + 1 < kTb) b[(t + 1) & 1] = load_halves(cur + (t + 1) * kTile, 1024);
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i][t] = mfma8<j>(a[j % kSets][i], b[t & 1], acc[i][t], sw[i], sx[t]);
        asm volatile("" ::: "memory");          // and an operand from LDS just before the products with the one before it
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (j == 2) put_scales(q + 1);
      // the copies for the next step have arrived when no more is on its way than the two steps after them asked for
      wait_loads<2 * (kCopies + 2 * RB)>();
      lds_barrier();
    }, std::make_integer_sequence<int, 4>{});
  }
  wait_loads<0>();      // no copy outlives the workgroup's LDS
  float* const slice = part ? part + (int64_t)blockIdx.y * M * w.N : nullptr;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t n = 16 * (int64_t)(rb0 + i) + 4 * g;
    if (n >= w.N) continue;
#pragma unroll
    for (int t = 0; t < kTb; ++t) {
      const int64_t m = m0 + 16 * t + r;
      if (m >= M) continue;
      if (!slice) {
        put4(y + m * ys + n, acc[i][t], w.N - n);
      } else {
        float* to = slice + m * w.N + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < w.N) to[e] = acc[i][t][e];
      }
    }
  }
}

// The splits' sums, added in their order.
__global__ __launch_bounds__(256) void k_join8(const float* part, int splits, int64_t M, int64_t N, _Float16* y,
                                               int64_t ys) {
  const int64_t all = M * N;
  for (int64_t o = (int64_t)blockIdx.x * 256 + threadIdx.x; o < all; o += (int64_t)gridDim.x * 256) {
    float v = part[o];
    for (int k = 1; k < splits; ++k) v += part[k * all + o];
    const int64_t m = o / N;
    y[m * ys + (o - m * N)] = (_Float16)v;
  }
}

template <int RB>
hipError_t go_tiled(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, float* part,
                    const Linear8Plan& p, hipStream_t s) {
  const int NT = (w.Nb + 4 * RB - 1) / (4 * RB), MT = (int)((M + 16 * kTb - 1) / (16 * kTb));
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_tiled8<RB>),
                                     hipFuncAttributeMaxDynamicSharedMemorySize, kTiledLds);
  if (e != hipSuccess) return e;
  k_tiled8<RB><<<dim3((unsigned)(NT * MT), (unsigned)p.splits), dim3(256), kTiledLds, s>>>(x, (int)M, w, y, ys, part, NT,
                                                                                           NT * MT, p.per);
  e = hipGetLastError();
  if (e == hipSuccess && part) {
    const int64_t groups = (M * w.N + 255) / 256;
    k_join8<<<dim3((unsigned)(groups < 8192 ? groups : 8192)), dim3(256), 0, s>>>(part, p.splits, M, w.N, y, ys);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

Linear8Plan plan_linear8(int64_t M, int64_t N, int64_t K) {
  Linear8Plan p = {};
  const int64_t Nb = (N + 15) / 16, Kt = (K + kQ8Block - 1) / kQ8Block, Kq = (Kt + 3) / 4;
  p.splits = 1;
  p.per = (int)(4 * Kq);
  if (M <= 64) {
    p.nt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    p.r = Nb >= 2048 ? 2 : 1;
    p.waves = (int)(Kq < 8 ? Kq : 8);
    p.groups = 2 * ((Nb + p.r - 1) / p.r);     // of 512 threads
    return p;
  }
  const int64_t MT = (M + 16 * kTb - 1) / (16 * kTb);
  p.r = ((Nb + 15) / 16) * MT >= 256 ? 4 : 2;
  const int64_t T = ((Nb + 4 * p.r - 1) / (4 * p.r)) * MT;
  if (T < 256) {
    int64_t S = 512 / T;
    S = S < Kq ? S : Kq;
    const int64_t per = (Kq + S - 1) / S;
    p.per = (int)(4 * per);
    p.splits = (int)((Kq + per - 1) / per);
    if (p.splits > 1) p.bytes = (size_t)p.splits * M * N * sizeof(float);
  }
  p.groups = T * p.splits;
  return p;
}

hipError_t launch_linear8(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, void* ws,
                          const Linear8Plan& p, hipStream_t s) {
  if (p.nt == 1) return p.r == 1 ? go_stream<1, 1>(x, M, w, y, ys, p, s) : go_stream<1, 2>(x, M, w, y, ys, p, s);
  if (p.nt == 2) return p.r == 1 ? go_stream<2, 1>(x, M, w, y, ys, p, s) : go_stream<2, 2>(x, M, w, y, ys, p, s);
  if (p.nt == 4) return p.r == 1 ? go_stream<4, 1>(x, M, w, y, ys, p, s) : go_stream<4, 2>(x, M, w, y, ys, p, s);
  float* part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  return p.r == 4 ? go_tiled<4>(x, M, w, y, ys, part, p, s) : go_tiled<2>(x, M, w, y, ys, part, p, s);
}

}  // namespace mq
