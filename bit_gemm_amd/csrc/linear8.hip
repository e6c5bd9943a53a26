// The product of 8-bit rows with 8-bit weights (include/mosaicq_head.h,
// mq_linear8):
//
//   Y[m][n] = sum over blocks b of 128 of 2^(ex[m][b] + ew[n][b]) sum_k x[m][k] w[n][k]
//
// on the fp8 matrix instruction of 128 columns, which takes both scales as
// exponent bytes and applies them itself. The weights are the A operand, so a
// lane holds four outputs of a token that follow each other. The instruction
// adds in groups of 8 columns, in which what lies below 2^-13 of the largest
// product is cut, and the groups in fp32. It has twice the rate of the fp16
// instruction, and what it cuts, at most 7 2^-13 of the groups' largest
// products, is 8 10^-5 of a sum of one sign over magnitudes of 2^12 and not seen
// beside fp16's rounding (4.9 10^-4) where signs are mixed; an fp32 output would
// hold no more, so there is none.
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

// Four outputs that follow each other, of which `left` exist: one store, which memory takes at any address.
__device__ __forceinline__ void put4(_Float16* y, float4_t v, int64_t left) {
  typedef _Float16 half4_any_t __attribute__((ext_vector_type(4), aligned(2)));
  if (left >= 4) {
    *reinterpret_cast<half4_any_t*>(y) = (half4_any_t){(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
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

// The codes of 16 tokens x 128 columns in LDS are filled by two copies of 1 KiB, in lane order. Copy u, lane l brings row
// 8 u + l / 8, chunk l % 8 ^ l / 8 of its 8 chunks of 16 bytes: eight lanes read a row's whole line (quads with runs of 64
// bytes ask for each line twice: X took twice the time of as many bytes of weights), and the 8 lanes that LDS serves at once
// when the operand is read back (rows n .. n + 7, one chunk) find 8 different banks of 16 bytes.
__device__ __forceinline__ uint32_t stage_from(int lane, uint32_t stride) {
  return (uint32_t)(lane >> 3) * stride + 16u * (uint32_t)((lane & 7) ^ (lane >> 3));
}
// Where lane n + 16 g finds chunk g of row n; chunk 4 + g lies 64 bytes away from it, up or down.
__device__ __forceinline__ uint32_t stage_pos(int lane) {
  const int n = lane & 15, g = lane >> 4;
  return 16u * (uint32_t)(8 * n + (g ^ (n & 7)));
}

// ------------------------------------------------------------ few tokens
// Up to 16 NT tokens: a workgroup takes R blocks of 16 weight rows, its waves
// fours of tiles along K in turn (a lane's scales of four blocks are one word).
// The weights go from memory straight to the registers that the instruction
// reads, once. The tokens' codes come from L2 through a part of LDS that is the
// wave's own: read in the operand's order they are 16 rows an instruction, in
// pieces of 16 bytes (16 tokens, 11008 x 4096: 12.1 us so, 10.0 through LDS).
// The waves' sums meet in LDS and are added in their order. Bound by the
// reading of the weights: 131072 x 4096, 16 tokens, 94 us (5.8 TB/s);
// 11008 x 4096, 16 tokens, 10.2 us (4.5); 4096 x 4096, one token, 4.3 us (3.9),
// of which 3 to begin and end. (Averages of traced calls.) Where a layer has few
// rows and a long K, the few workgroups are what binds: 128 x 16384, 16 tokens,
// 6.6 us for 2 MB on 8 CUs; 128 x 65536 20 us.
template <int NT, int R>
__global__ __launch_bounds__(512) void k_stream8(Rows8 x, int M, W8 w, _Float16* y, int64_t ys) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int waves = blockDim.x >> 6;
  const int r = lane & 15;
  const int rb0 = blockIdx.x * R;
  uint8_t* const own = lds + wave * (4 * NT * kTile);
  const __amdgpu_buffer_rsrc_t xr =      // reads past the tokens' rows give zero
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(x.codes), 0, (int)(M * x.stride), kBufferRaw);
  const uint32_t xl = stage_from(lane, (uint32_t)x.stride);
  const uint8_t* xs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xs[t] = x.scales + (int64_t)min(16 * t + r, M - 1) * x.sstride;
  const uint32_t pos = stage_pos(lane), pos4 = pos ^ 64;
  float4_t acc[R][NT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};

  for (int q = wave; q < w.Kq; q += waves) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              xr, (__attribute__((address_space(3))) void*)(own + (j * NT + t) * kTile + 1024 * u), 16,
              xl + (uint32_t)(16 * t + 8 * u) * (uint32_t)x.stride + (uint32_t)(min(4 * q + j, w.Kt - 1) * kQ8Block), 0, 0, 0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    int sw[R], sx[NT];
    i32x8_t a[4][R];
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
    for (int t = 0; t < NT; ++t) sx[t] = row_scales(xs[t], q, w.Kt);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(8 * R) : "memory");      // the copies, which were asked for before 8 R loads
    four([&](auto j) {
      if (4 * q + j < w.Kt) {
        i32x8_t b[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint8_t* const from = own + (j * NT + t) * kTile;
          b[t] = join(*reinterpret_cast<const i32x4_t*>(from + pos), *reinterpret_cast<const i32x4_t*>(from + pos4));
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[i][t] = mfma8<j>(a[j][i], b[t], acc[i][t], sw[i], sx[t]);
      }
    }, std::make_integer_sequence<int, 4>{});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");                // before the next copies land where these were read
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  float4_t* const red = reinterpret_cast<float4_t*>(lds);
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
  const int lds = p.waves * 4 * NT * kTile;      // the tokens' codes, later the sums (R is 2 at most)
  static_assert(R * 1024 <= 4 * kTile, "the sums of a wave fit where its codes were");
  hipError_t e = hipSuccess;
  if (lds > 65536)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_stream8<NT, R>), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  k_stream8<NT, R><<<dim3((unsigned)((w.Nb + R - 1) / R)), dim3(64 * p.waves), lds, s>>>(x, (int)M, w, y, ys);
  return hipGetLastError();
}

// ----------------------------------------------------------- many tokens
// A workgroup of 4 waves makes 64 RB weight rows x 16 TB tokens; a wave its own
// 16 RB rows with all the tokens. The weights lie in the instruction's order,
// so they go from L2 straight to registers; the tokens' codes go to LDS, where
// the waves share them, by direct copies three blocks of 128 columns ahead
// (one ahead, with conditions in a step and scales straight from memory, 2048
// tokens took 505 us at 28672 x 8192, and about 440 so). Steps are taken by
// fours, which share the words of scales; what lies past K in the last four is
// zero in LDS and adds nothing. Nothing in a step is under a condition: a load
// there would be waited for where the branches meet.
// What it spends its time on, by the same kernel with parts left out (us; whole,
// without loads in the loop, without products, without either, and with the same
// four tiles asked for again and again, so that little comes from beyond L2):
//   28672 x 8192, 2048 tokens  440 (2.2 PFLOP/s)  276  381  168  389
//   4096 x 14336, 512 tokens   42 (1.4; 55 where the weights come from HBM)  28  49  32  37
//   10007 x 2501, 333 tokens   18 (0.9)  13.5  18  14  16.5
// Much work: the loads through L2, which the products cover in part; what lies
// beyond L2 is an eighth. One round of tiles: mostly a step by itself, its LDS
// reads, products and barrier with one workgroup of four waves a CU. (Without
// products, what takes their place to use the operands costs some time.) Tiles of
// 256 x 256 by 8 waves leave one workgroup a CU and were slower.
// codes; scales of the tokens, 8 blocks of each, and of the weight rows, 4 of each; each twice
constexpr int tiled_lds(int rb, int tokens) { return 4 * tokens * kQ8Block + 2 * (8 * tokens + 4 * 64 * rb); }

// Waits until no more than N loads are on their way, and for the wave's own LDS accesses, then for the other waves. (A fence
// would wait for every copy into LDS, also for those that the next steps need.)
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int RB, int TB>
__global__ __launch_bounds__(256, 2) void k_tiled8(Rows8 x, int M, W8 w, _Float16* y, int64_t ys, float* part, int NT,
                                                   int T, int per) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int kAhead = RB == 4 ? 1 : 3;      // steps that the weights are asked for ahead: what the registers hold
  constexpr int kSets = kAhead + 1;
  constexpr int kCopies = TB / 2;              // of a wave in a step
  constexpr int kTokens = 16 * TB, kRows = 64 * RB, kStage = kTokens * kQ8Block;
  uint2* const token_scales = reinterpret_cast<uint2*>(lds + 4 * kStage);
  uint32_t* const row_scale_words = reinterpret_cast<uint32_t*>(lds + 4 * kStage + 2 * 8 * kTokens);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, g = lane >> 4;
  const int tile = xcd_tile(blockIdx.x, T), MT = T / NT;
  const int nt = tile / MT, mt = tile - nt * MT;
  const int rb0 = (nt * 4 + wave) * RB, m0 = kTokens * mt;
  const int kt0 = blockIdx.y * per, kt1 = min(w.Kt, kt0 + per), q1 = (kt1 + 3) >> 2;

  // the workgroup's token rows; reads past them give zero
  const int rows = min(kTokens, M - m0);
  const uint32_t range = (uint32_t)rows * (uint32_t)x.stride;
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(x.codes + (int64_t)m0 * x.stride), 0, (int)range, kBufferRaw);
  const uint32_t xl = stage_from(lane, (uint32_t)x.stride);
  auto copy = [&](int stage, int kt) {
    const uint32_t at = kt < kt1 ? (uint32_t)kt * kQ8Block : 0x40000000u;      // past the split: zero
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int tb = (4 * i + wave) >> 1, u = wave & 1;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (__attribute__((address_space(3))) void*)(lds + stage * kStage + tb * kTile + 1024 * u), 16,
          xl + (uint32_t)(16 * tb + 8 * u) * (uint32_t)x.stride + at, 0, 0, 0);
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
  // The scales: a thread asks for 8 of a token's at a time, once in 8 steps (128 tokens are 128 lines: asked for by fours
  // they were a sixth of all that came from L2; 16 at a time spilled registers that had to wait for them), and for a word of
  // a weight row's, four of them, once in 4; into LDS later. A token's 8 bytes are taken from where they lie, or, where that
  // would pass the end of all scales, from some bytes before and shifted; bytes past the row count as 127 (their codes are
  // zero, but a NaN there would not be).
  const uint8_t* const xs = x.scales + (int64_t)m0 * x.sstride;
  const int xs_own = min(tid % kTokens, M - 1 - m0) * (int)x.sstride;
  const int xs_last = (int)min((int64_t)0x40000000, (M - 1 - m0) * x.sstride + w.Kt - 8);
  const __amdgpu_buffer_rsrc_t wsr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(w.scales + (int64_t)64 * min(nt * 4 * RB, w.Nb - 1) * w.Kq), 0, 0x7FFFFFFF, kBufferRaw);
  const int ws_own = 64 * min(tid % kRows >> 4, w.Nb - 1 - min(nt * 4 * RB, w.Nb - 1)) * w.Kq + 4 * (tid & 15);
  uint64_t token_bytes;
  uint32_t row_word;
  auto token_over = [&](int q) { return max(0, xs_own + 4 * min(q, w.Kq - 1) - xs_last); };
  auto ask_token_scales = [&](int q) {
    typedef uint64_t u64_any_t __attribute__((aligned(1)));
    token_bytes = *reinterpret_cast<const u64_any_t*>(xs + (xs_own + 4 * min(q, w.Kq - 1) - token_over(q)));
  };
  auto put_token_scales = [&](int buffer, int q) {
    const uint64_t v = token_bytes >> (8 * token_over(q));
    const int have = min(w.Kt - 4 * min(q, w.Kq - 1), 8);
    const uint64_t own = ~0ull >> (8 * (8 - have)), u = (v & own) | (0x7F7F7F7F7F7F7F7Full & ~own);
    token_scales[buffer * kTokens + tid % kTokens] = make_uint2((uint32_t)u, (uint32_t)(u >> 32));
  };
  auto ask_row_scales = [&](int q) { row_word = __builtin_amdgcn_raw_buffer_load_b32(wsr, ws_own, 64 * min(q, w.Kq - 1), 0); };
  auto put_row_scales = [&](int q) { row_scale_words[(q & 1) * kRows + tid % kRows] = row_word; };

  float4_t acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[i][t] = float4_t{0.f, 0.f, 0.f, 0.f};

  const int q0 = kt0 >> 2;
  ask_token_scales(q0);
  ask_row_scales(q0);
#pragma unroll
  for (int j = 0; j < 3; ++j) copy(j, kt0 + j);
#pragma unroll
  for (int j = 0; j < kAhead; ++j) weights(j, kt0 + j);
  put_token_scales(0, q0);
  put_row_scales(q0);
  wait_and_meet<0>();
  const uint32_t pos = stage_pos(lane), pos4 = pos ^ 64;
  auto operand = [&](const uint8_t* p) {
    return join(*reinterpret_cast<const i32x4_t*>(p + pos), *reinterpret_cast<const i32x4_t*>(p + pos4));
  };
  for (int q = q0, buffer = 0; q < q1; buffer ^= 1) {
    const int qe = min(q + 2, q1), qs = q;
    ask_token_scales(qe);
    for (; q < qe; ++q) {
      const uint32_t* const ts = reinterpret_cast<const uint32_t*>(token_scales + buffer * kTokens + r) + (q - qs);
      const uint32_t* const rs = row_scale_words + (q & 1) * kRows + 16 * wave * RB + r;
      int sw[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) sw[i] = (int)rs[16 * i];
      ask_row_scales(q + 1);
      four([&](auto j) {
        const int kt = 4 * q + j;
        weights((j + kAhead) % kSets, kt + kAhead);     // before the copies: loads come back in order, and these are due first
        __builtin_amdgcn_sched_barrier(0);
        copy((j + 3) & 3, kt + 3);
        __builtin_amdgcn_sched_barrier(0);        // the loads go out first,
        const uint8_t* const cur = lds + j * kStage;
        i32x8_t b[2];
        int sx[2];
        b[0] = operand(cur);
        sx[0] = (int)ts[0];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
          if (t + 1 < TB) {
            b[(t + 1) & 1] = operand(cur + (t + 1) * kTile);
            sx[(t + 1) & 1] = (int)ts[32 * (t + 1)];
          }
#pragma unroll
          for (int i = 0; i < RB; ++i) acc[i][t] = mfma8<j>(a[j % kSets][i], b[t & 1], acc[i][t], sw[i], sx[t & 1]);
          asm volatile("" ::: "memory");          // and an operand from LDS just before the products with the one before it
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (j == 2) put_row_scales(q + 1);
        // the copies for the next step have arrived when no more is on its way than the two steps after them asked for
        wait_and_meet<2 * (kCopies + 2 * RB)>();
      }, std::make_integer_sequence<int, 4>{});
    }
    put_token_scales(buffer ^ 1, q);
    wait_and_meet<2 * (kCopies + 2 * RB)>();
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // no copy outlives the workgroup's LDS
  float* const slice = part ? part + (int64_t)blockIdx.y * M * w.N : nullptr;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t n = 16 * (int64_t)(rb0 + i) + 4 * g;
    if (n >= w.N) continue;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
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

// The splits' sums, added in their order: a workgroup takes 1024 outputs of a token.
__global__ __launch_bounds__(256) void k_join8(const float* part, int splits, int64_t M, int64_t N, int per_row,
                                               _Float16* y, int64_t ys) {
  const int64_t m = blockIdx.x / per_row, n = 1024 * (int64_t)(blockIdx.x - m * per_row) + 4 * (int)threadIdx.x;
  if (n >= N) return;
  typedef float float4_any_t __attribute__((ext_vector_type(4), aligned(4)));
  const float* p = part + m * N + n;
  float4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < splits; ++k, p += M * N) {
    if (n + 4 <= N) {
      v += *reinterpret_cast<const float4_any_t*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) v[i] += p[i];
    }
  }
  put4(y + m * ys + n, v, N - n);
}

template <int RB, int TB>
hipError_t go_tiled(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, float* part,
                    const Linear8Plan& p, hipStream_t s) {
  constexpr int kTokens = 16 * TB, kLds = tiled_lds(RB, kTokens);
  const int NT = (w.Nb + 4 * RB - 1) / (4 * RB), MT = (int)((M + kTokens - 1) / kTokens);
  hipError_t e = hipSuccess;
  if (kLds > 65536)
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(&k_tiled8<RB, TB>), hipFuncAttributeMaxDynamicSharedMemorySize,
                            kLds);
  if (e != hipSuccess) return e;
  k_tiled8<RB, TB><<<dim3((unsigned)(NT * MT), (unsigned)p.splits), dim3(256), kLds, s>>>(x, (int)M, w, y, ys, part, NT,
                                                                                        NT * MT, p.per);
  e = hipGetLastError();
  if (e == hipSuccess && part) {
    const int per_row = (int)((w.N + 1023) / 1024);
    k_join8<<<dim3((unsigned)(M * per_row)), dim3(256), 0, s>>>(part, p.splits, M, w.N, per_row, y, ys);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t launch_linear8(const Rows8& x, int64_t M, const W8& w, _Float16* y, int64_t ys, void* ws,
                          const Linear8Plan& p, hipStream_t s) {
  if (p.nt == 1) return p.r == 1 ? go_stream<1, 1>(x, M, w, y, ys, p, s) : go_stream<1, 2>(x, M, w, y, ys, p, s);
  if (p.nt == 2) return p.r == 1 ? go_stream<2, 1>(x, M, w, y, ys, p, s) : go_stream<2, 2>(x, M, w, y, ys, p, s);
  float* part = p.splits > 1 ? static_cast<float*>(ws) : nullptr;
  switch (16 * p.r + p.tb) {
    case 16 * 4 + 8: return go_tiled<4, 8>(x, M, w, y, ys, part, p, s);
    case 16 * 2 + 8: return go_tiled<2, 8>(x, M, w, y, ys, part, p, s);
    case 16 * 2 + 4: return go_tiled<2, 4>(x, M, w, y, ys, part, p, s);
    case 16 * 2 + 2: return go_tiled<2, 2>(x, M, w, y, ys, part, p, s);
    case 16 * 1 + 4: return go_tiled<1, 4>(x, M, w, y, ys, part, p, s);
    default: return go_tiled<1, 2>(x, M, w, y, ys, part, p, s);
  }
}

}  // namespace mq
