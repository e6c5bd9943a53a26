/*
 * mosaicq_block.h -- C ABI of the operators that stand between the 4-bit
 * linears of a decoder block (mosaicq.h) when it serves: rotary positions,
 * the append to a key/value cache held in 8 bits, the attention that reads
 * that cache, and the norms before and after a block with its gate and
 * residual, also with an output in 8 bits. Library: libmosaicq_block.so, which stands beside libmosaicq.so
 * and needs nothing of it (mq_status is shared).
 *
 * Conventions, as in mosaicq.h: pointers named *_dev (and every pointer in
 * the structs below) are device pointers on the device that is current when
 * the call is made and stay owned by the caller; hip_stream is a hipStream_t
 * (NULL = the default stream); work is enqueued on it in order and no call
 * synchronises, allocates device memory or keeps anything between calls, so
 * every call may be captured into a HIP graph; nothing throws across the ABI;
 * arguments are checked before any HIP call is made. Activations are fp16,
 * as the linears read and write them; sums, softmax statistics and norms are
 * held in fp32. Strides count elements.
 *
 * Sizes that live on the device (lengths, tables, positions) cannot be
 * checked by the host: the kernels clamp them to the arrays' bounds, so a
 * wrong value gives wrong or NaN outputs but no access outside the arrays.
 */
#ifndef MOSAICQ_BLOCK_H
#define MOSAICQ_BLOCK_H

#include "mosaicq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary
 * Position p turns pair i of a head by the angle p f_i:
 *   y_a = x_a c - x_b s,  y_b = x_b c + x_a s,  (c, s) = m (cos, sin)(p f_i),
 * f_i = theta^(-2 i / rot_dim), i < rot_dim / 2. The pair is (i, i + rot_dim/2)
 * in the half layout, (2 i, 2 i + 1) in the interleaved one; elements
 * from rot_dim on pass unchanged. Scaled positions, for contexts longer than
 * the original one:
 *   MQ_ROPE_LINEAR  f_i / factor
 *   MQ_ROPE_BASE    theta * factor^(rot_dim / (rot_dim - 2)) in place of theta
 *   MQ_ROPE_PARTS   (the YaRN rule, Peng et al. 2023) f_i (1 - r_i) + f_i r_i / factor with
 *                   r_i = clamp((i - lo) / (hi - lo), 0, 1), where lo and hi are the pairs that
 *                   turn `turns_fast` and `turns_slow` times in `original` positions
 *                   (rot_dim ln(original / (2 pi turns)) / (2 ln theta), rounded down and up and
 *                   clamped to [0, rot_dim - 1]); and m = 0.1 ln(factor) + 1 (m = 1 elsewhere)
 */
typedef enum { MQ_ROPE_HALF = 0, MQ_ROPE_INTERLEAVED = 1 } mq_rope_layout;
typedef enum { MQ_ROPE_NONE = 0, MQ_ROPE_LINEAR = 1, MQ_ROPE_BASE = 2, MQ_ROPE_PARTS = 3 } mq_rope_scaling;

typedef struct {
  int32_t rot_dim;      /* rotated elements of a head, even, 2 .. 1024 */
  int32_t scaling;      /* mq_rope_scaling */
  double theta;         /* > 1 */
  double factor;        /* >= 1 (not read for MQ_ROPE_NONE) */
  double original;      /* MQ_ROPE_PARTS: the original context, > 0 */
  double turns_fast;    /* MQ_ROPE_PARTS: commonly 32 */
  double turns_slow;    /* MQ_ROPE_PARTS: commonly 1, < turns_fast */
} mq_rope_spec;

/*
 * mq_rope_table -- cos and sin of positions 0 .. positions - 1, computed in
 * 64 bits and rounded once to fp32, so that the angle stays exact however far
 * the position: table_dev_f32 [positions, rot_dim / 2, 2] (cos, sin), 8-byte
 * aligned, written whole. Errors: MQ_ERR_INVALID_ARG (NULL or misaligned
 * pointer, a field out of the ranges above, positions <= 0),
 * MQ_ERR_UNSUPPORTED (positions * rot_dim >= 2^31), MQ_ERR_DEVICE.
 */
mq_status mq_rope_table(const mq_rope_spec* spec, int64_t positions, float* table_dev_f32, void* hip_stream);

/* A table with what is needed to use it. */
typedef struct {
  const float* table;   /* from mq_rope_table */
  int64_t positions;    /* its rows */
  int32_t rot_dim;
  int32_t layout;       /* mq_rope_layout */
} mq_rope_plan;

/*
 * mq_rope -- rotate the heads of `tokens` tokens.
 *
 *   X_dev_fp16   [tokens, heads, head_dim], element (t, h, d) at
 *                t * x_token_stride + h * x_head_stride + d
 *   pos_dev_i32  [tokens] position of each token; a token whose position lies
 *                outside the table gets NaN in its rotated elements
 *   rope         table, rotated elements (<= head_dim) and layout
 *   inverse      0, or 1 to turn back (the transpose, which is also the
 *                gradient; where the scaling has m != 1, m multiplies again)
 *   Y_dev_fp16   as X with its own strides; Y may be X with X's strides
 *   tokens >= 0 (0 enqueues nothing; arguments are checked all the same), heads
 *   >= 1, head_dim >= 2; pointers not NULL, 2-byte aligned
 *
 * Products and sums are rounded one by one in fp32, the result once to fp16.
 * Errors: MQ_ERR_INVALID_ARG, MQ_ERR_UNSUPPORTED (tokens or heads * head_dim
 * >= 2^31), MQ_ERR_DEVICE.
 */
mq_status mq_rope(const void* X_dev_fp16, int64_t tokens, int32_t heads, int32_t head_dim, int64_t x_token_stride,
                  int64_t x_head_stride, const int32_t* pos_dev_i32, const mq_rope_plan* rope, int32_t inverse,
                  void* Y_dev_fp16, int64_t y_token_stride, int64_t y_head_stride, void* hip_stream);

/* ------------------------------------------------------------------- cache
 * Tokens are cached in blocks of 64. A block that is full holds 8-bit codes
 * with one fp32 scale for each kv head, of its keys and of its values:
 *   scale = max |x| / M over the head's 64 x head_dim elements, M = 127 (int8)
 *   or 448 (OCP e4m3); code = round to nearest even of x i, whole numbers clamped
 *   to -127 .. 127 or e4m3, with i = M (1 / max |x|), each of these fp32 steps
 *   rounded; all 0 where max |x| = 0.
 * A sequence's last block, while it is not full, stays in fp16 in the
 * sequence's slot of the tails, and is coded once, when its last token
 * arrives: codes do not depend on how the tokens arrived, and no code is
 * ever rounded twice. A key or value vector of a token (in one kv head) with
 * an Inf or NaN element makes NaN every output that attends to it; once its
 * block is coded, every output of that kv head that attends to any token of
 * the block. No other output is touched.
 */
enum { MQ_KV_BLOCK = 64 };
typedef enum { MQ_KV_INT8 = 0, MQ_KV_E4M3 = 1 } mq_kv_format;

typedef struct {
  void* k_codes;        /* [num_blocks, kv_heads, 64, head_dim] bytes, 16-byte aligned */
  void* v_codes;        /* [num_blocks, kv_heads, head_dim, 64] bytes, 16-byte aligned */
  float* k_scale;       /* [num_blocks, kv_heads] */
  float* v_scale;       /* [num_blocks, kv_heads] */
  void* k_tail;         /* [num_slots, kv_heads, 64, head_dim] fp16, 16-byte aligned */
  void* v_tail;         /* [num_slots, kv_heads, head_dim, 64] fp16, 16-byte aligned */
  int64_t num_blocks;   /* >= 1 */
  int64_t num_slots;    /* >= 1 */
  int32_t kv_heads;     /* 1 .. 1024 */
  int32_t head_dim;     /* 64 or 128 */
  int32_t format;       /* mq_kv_format */
} mq_kv_cache;

/* The sequences of one step. Sequence s brings the tokens cu_q[s] .. cu_q[s + 1] - 1
 * (rows of q, k, v and of the output), which are the last ones of its
 * kv_len[s] tokens: new token i has position kv_len[s] - n + i. */
typedef struct {
  const int32_t* cu_q;          /* [seqs + 1], 0 .. tokens, not descending */
  const int32_t* kv_len;        /* [seqs] tokens of the sequence, the new ones counted */
  const int32_t* block_table;   /* [seqs, table_width] the sequence's blocks, in order */
  const int32_t* slots;         /* [seqs] the sequence's tail slot, all different; NULL: sequence s has slot s */
  int64_t seqs;                 /* >= 0; at most 65535 */
  int64_t tokens;               /* rows of q, k, v; >= 0 */
  int64_t table_width;          /* >= 1 */
  int64_t max_new;              /* at least the most new tokens of a sequence, >= 1 */
  int64_t max_len;              /* at least the longest kv_len, >= 1 */
} mq_kv_batch;

/*
 * mq_kv_append -- write the new tokens' keys and values into the cache, with
 * the rotation of keys and queries in the same launch.
 *
 *   q_dev_fp16    [tokens, q_heads, head_dim], rows q_stride apart; read only
 *                 with a rope plan; NULL leaves the queries alone
 *   k_, v_dev_fp16  [tokens, kv_heads, head_dim], rows k_stride, v_stride apart
 *                 (so a joined q + k + v projection is read where it lies)
 *   rope          NULL (keys are stored as they are), or a plan with rot_dim
 *                 <= head_dim: queries and keys are turned to their positions
 *                 (rounded to fp16, as mq_rope) before they are written
 *   q_out_dev_fp16  [tokens, q_heads, head_dim], rows q_out_stride apart; may
 *                 be q itself; needed when q and rope are given
 *
 * Blocks that the new tokens fill are coded into block_table's blocks; the
 * tokens of a block that stays open go into the tail; nothing else of the
 * cache is written. Appending the same token again at the same position
 * gives the same cache while its block is open. Tokens with a negative
 * position, of a block past table_width, or whose block or slot is out of
 * range are dropped. Errors: MQ_ERR_INVALID_ARG, MQ_ERR_UNSUPPORTED (head_dim
 * not 64 or 128, more than 2^31 - 1 tokens, bounds of 2^24 workgroups or more:
 * seqs * kv_heads * (max_new + 126) / 64, and seqs * (max_new + 3) / 4 where
 * queries are turned), MQ_ERR_DEVICE.
 */
mq_status mq_kv_append(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q_dev_fp16, int32_t q_heads,
                       int64_t q_stride, const void* k_dev_fp16, int64_t k_stride, const void* v_dev_fp16,
                       int64_t v_stride, const mq_rope_plan* rope, void* q_out_dev_fp16, int64_t q_out_stride,
                       void* hip_stream);

/*
 * mq_kv_attention -- O = softmax(scale q K^T) V over each sequence's cache.
 * Query head h reads kv head h / (q_heads / kv_heads). With causal != 0 new
 * token i attends to the positions up to its own, kv_len - n + i, else to all
 * kv_len; a query with nothing to attend to gets zeros, one with an Inf or NaN
 * element that attends to anything NaN.
 *
 *   q_dev_fp16    [tokens, q_heads, head_dim], rows q_stride apart, 16-byte
 *                 aligned (pointer and stride)
 *   q_heads       a multiple of kv_heads, at most 64 for each kv head
 *   scale         multiplies the scores (commonly head_dim^-1/2), finite
 *   out_dev_fp16  [tokens, q_heads, head_dim], rows out_stride apart, 8-byte
 *                 aligned; written for every token of a sequence, rows of none
 *                 (before cu_q[0], from cu_q[seqs] on) are left as they are; not q
 *   workspace_dev, workspace_bytes  fp32 partial results, at least
 *                 mq_kv_attention_workspace bytes (0: NULL is accepted),
 *                 16-byte aligned; calls that overlap in time need their own
 *
 * The same call gives the same bits: work split over a long cache is joined
 * in a fixed order. Errors: MQ_ERR_INVALID_ARG (also a workspace that is too
 * small), MQ_ERR_UNSUPPORTED (head_dim, more than 64 query heads for a kv
 * head, bounds that need 2^32 threads or more: 2 for each of seqs * max_new *
 * q_heads rows, 256 for each sequence's kv head at least, and where a long cache
 * is split 256 for each token's query head), MQ_ERR_DEVICE.
 */
mq_status mq_kv_attention(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q_dev_fp16, int32_t q_heads,
                          int64_t q_stride, int32_t causal, float scale, void* out_dev_fp16, int64_t out_stride,
                          void* workspace_dev, size_t workspace_bytes, void* hip_stream);

/* mq_kv_attention_workspace -- bytes that mq_kv_attention needs for a batch of
 * these sizes (by seqs, tokens, max_new and max_len; no pointer is read). */
mq_status mq_kv_attention_workspace(const mq_kv_cache* cache, const mq_kv_batch* batch, int32_t q_heads,
                                    size_t* bytes);

/* ------------------------------------------------------------------- norms
 * mq_norm_residual -- what stands between two blocks, in one pass:
 *   r' = alpha r + beta g (y / rms(y)) (w_post + o)      the branch joins the residual
 *   h  = (r' / rms(r')) (w_pre + o)                      the next block's input
 * with rms(x) = sqrt(mean(x^2) + eps) over a row, g the gate. Without w_post
 * the branch joins as it is (r' = alpha r + beta g y); without a gate g = 1;
 * without y, r' = r and only h is written; without w_pre only r' is. h is
 * taken from r' as it is stored, so that a later norm of the stored residual
 * gives the same. Statistics and products in fp32.
 */
typedef struct {
  const void* y;         /* [tokens, width] fp16 block output, rows y_stride apart; NULL: none */
  const void* r;         /* [tokens, width] residual, fp16 or fp32, rows r_stride apart */
  const void* gate;      /* [tokens, width] fp16, rows gate_stride apart (0: one row for all tokens); NULL: 1 */
  const void* w_post;    /* [width] fp16, or NULL */
  const void* w_pre;     /* [width] fp16, or NULL */
  void* r_out;           /* as r, rows r_out_stride apart; may be r; needed with y */
  void* h_out;           /* [tokens, width] fp16, rows h_stride apart; needed with w_pre */
  int64_t tokens;        /* >= 0 */
  int64_t width;         /* 1 .. 65536 */
  int64_t y_stride, r_stride, gate_stride, r_out_stride, h_stride;
  float alpha, beta, eps, weight_offset;   /* eps >= 0; weight_offset is o above */
  int32_t residual_fp32; /* 0: r and r_out are fp16, 1: fp32 */
} mq_norm_args;

/* Errors: MQ_ERR_INVALID_ARG (NULL where needed, sizes out of range, strides
 * below width, misaligned elements, a scalar that is not finite),
 * MQ_ERR_UNSUPPORTED (width > 65536, tokens >= 2^31), MQ_ERR_DEVICE. */
mq_status mq_norm_residual(const mq_norm_args* args, void* hip_stream);

/*
 * mq_norm_residual_q8 -- mq_norm_residual with h as 8-bit rows, for the linears
 * that take them (mosaicq_head.h): r' is the same bits, and h, before it is
 * rounded to fp16, is coded as mq_quantize8 codes (OCP e4m3 codes with a
 * power-of-two scale for each block of 128 elements, rounded once).
 *
 *   args         as above with w_pre; h_out is the codes, [tokens, K8] bytes,
 *                K8 = 128 ceil(width / 128), 16-byte aligned, rows h_stride bytes
 *                apart (>= K8, a multiple of 16); bytes past width, up to K8, are 0,
 *                in a block with an Inf or NaN 127 (NaN) like its other codes
 *   scales_dev   [tokens, K8 / 128] bytes, rows scales_stride bytes apart
 *
 * Errors as mq_norm_residual, and MQ_ERR_INVALID_ARG without w_pre.
 */
mq_status mq_norm_residual_q8(const mq_norm_args* args, void* scales_dev, int64_t scales_stride, void* hip_stream);

#ifdef __cplusplus
}
#endif
#endif /* MOSAICQ_BLOCK_H */
