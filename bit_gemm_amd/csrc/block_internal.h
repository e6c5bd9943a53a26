// Internal declarations of the block operators (include/mosaicq_block.h):
// what the host hands to the kernels, and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/mosaicq_block.h"

namespace mq {

constexpr int kKvBlock = MQ_KV_BLOCK;

struct RopeView {
  const float2* table;   // [positions][rot / 2] (cos, sin); NULL: no rotation
  int64_t positions;
  int rot;
  int interleaved;
};

struct KvView {
  uint8_t *kc, *vc;
  float *ks, *vs;
  _Float16 *kt, *vt;
  int64_t blocks;
  int slots;
  int hk;
};

struct BatchView {
  const int32_t *cu, *len, *table, *slot;
  int seqs, tokens, width;
  int max_new, max_len;
};

// Rows of a [tokens, heads, head_dim] tensor, `stride` elements apart.
struct RowsIn {
  const _Float16* p;
  int64_t stride;
};
struct RowsOut {
  _Float16* p;
  int64_t stride;
};

hipError_t launch_rope_table(const double* freq, int pairs, double mag, int64_t positions, float2* table,
                             hipStream_t s);
hipError_t launch_rope(const _Float16* x, int64_t tokens, int heads, int dim, int64_t xt, int64_t xh,
                       const int32_t* pos, const RopeView& rope, int inverse, _Float16* y, int64_t yt, int64_t yh,
                       hipStream_t s);
// grid_too_large: set where the launch would have too many threads (nothing is enqueued then)
hipError_t launch_kv_append(const KvView& kv, int dim, int format, const BatchView& b, RowsIn q, int hq, RowsIn k,
                            RowsIn v, const RopeView& rope, RowsOut qo, bool* grid_too_large, hipStream_t s);

// Query rows a workgroup of the kernel for many rows holds: 32 a wave, 8 waves, and one workgroup a CU; for heads of 64
// elements 4 waves and two workgroups a CU, which even out better (5 pieces: 105 us against 115; with heads of 128 the
// codes laid twice as often cost more: a prompt of 4096 164 us against 150).
constexpr int attn_rows(int dim) { return dim == 64 ? 128 : 256; }


// A launch takes fewer than 2^32 threads.
inline bool launchable(int64_t groups, int threads) { return groups < (int64_t(1) << 32) / threads; }

// How the attention of a batch is run: a rule on sizes alone (kv_attn.hip).
struct AttnPlan {
  int nt;             // blocks of 16 query rows a workgroup holds; 0: the kernel for many rows, attn_rows of them
  int row_tiles;      // row tiles of the sequence with the most rows
  bool slices;        // many rows: a workgroup takes a slice of all the work, whatever row tiles that is of
  int chunk;          // else: cache blocks of one workgroup
  int splits;         // and workgroups along the cache of the longest sequence; 1: no workspace
  int64_t groups;     // workgroups in all
  int threads;        // of each
  int64_t joins;      // workgroups of 256 threads that join the splits
  size_t bytes;       // workspace
};
AttnPlan plan_attention(int hk, int hq, int dim, int64_t seqs, int64_t tokens, int64_t max_new, int64_t max_len);
hipError_t launch_kv_attention(const KvView& kv, int dim, int format, const BatchView& b, RowsIn q, int hq, int causal,
                               float scale, RowsOut out, void* ws, const AttnPlan& plan, hipStream_t s);

hipError_t launch_norm_residual(const mq_norm_args& a, hipStream_t s);

}  // namespace mq
