/*
 * mosaicq_head.h -- C ABI of the way out of a model: the linear of 8-bit rows
 * with 8-bit weights (the head's product, or any layer that is not held in
 * 4 bits) and the sampling of a token from its logits. Library:
 * libmosaicq_head.so, which stands beside libmosaicq.so and needs nothing of
 * it (mq_status is shared). mq_norm_residual_q8 (mosaicq_block.h) makes the
 * rows that mq_linear8 reads.
 *
 * Conventions, as in mosaicq_block.h: pointers named *_dev (and every pointer
 * in the structs below) are device pointers on the device that is current
 * when the call is made and stay owned by the caller; hip_stream is a
 * hipStream_t (NULL = the default stream); work is enqueued on it in order
 * and no call synchronises, allocates device memory or keeps anything between
 * calls, so every call may be captured into a HIP graph; nothing throws
 * across the ABI; arguments are checked before any HIP call is made. Outputs
 * do not overlap inputs or each other. The same call gives the same bits.
 *
 * 8-bit rows. A row of K values is held as K8 = 128 ceil(K / 128) OCP e4m3
 * codes (0 past K) and a scale for each block of 128, a power of two 2^e held
 * as the byte e + 127 (e8m0): e is the smallest whole number >= -127 with
 * max |x| <= 448 2^e over the block, 0 where the block is all zero;
 * code = x 2^-e rounded to nearest even. A power of two rounds nothing, and
 * the matrix instruction applies it by itself. A block with an Inf or NaN has
 * the scale byte 255 (NaN) and NaN codes (127, also past K).
 */
#ifndef MOSAICQ_HEAD_H
#define MOSAICQ_HEAD_H

#include "mosaicq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * mq_quantize8 -- fp16 rows as 8-bit rows.
 *
 *   X_dev_fp16   [M, K], rows x_stride elements apart (>= K), 2-byte aligned
 *   M, K         M >= 0 (0 enqueues nothing), K in 1 .. 2^20
 *   codes_dev    [M, K8] bytes, rows codes_stride bytes apart (>= K8, a
 *                multiple of 16), 16-byte aligned; K8 bytes of a row are written
 *   scales_dev   [M, K8 / 128] bytes, rows scales_stride bytes apart (>= K8 / 128)
 *
 * Errors: MQ_ERR_INVALID_ARG, MQ_ERR_UNSUPPORTED (K > 2^20, M >= 2^31,
 * M * K8 >= 2^42), MQ_ERR_DEVICE.
 */
mq_status mq_quantize8(const void* X_dev_fp16, int64_t M, int64_t K, int64_t x_stride, void* codes_dev,
                       int64_t codes_stride, void* scales_dev, int64_t scales_stride, void* hip_stream);

/* Weights [N, K] as 8-bit rows, in the order in which the matrix cores take
 * them. With Nb = ceil(N / 16), Kt = ceil(K / 128) and Kq = ceil(Kt / 4):
 *   codes   [Nb, Kt, 2, 64, 16] bytes: byte b of lane l, half h of a tile is the
 *           code of row 16 rb + l % 16, column 128 kt + 64 h + 16 (l / 16) + b;
 *           rows past N and columns past K hold 0
 *   scales  [Nb, Kq, 16, 4] bytes: byte j of row r is the scale byte of row
 *           16 rb + r, block 4 q + j; 127 past N and past Kt
 * so that a wave's loads are whole runs of memory. */
typedef struct {
  void* codes;          /* mq_pack8_bytes gives the bytes of both; 16-byte aligned */
  void* scales;         /* 4-byte aligned */
  int64_t N, K;
} mq_w8;

/* mq_pack8_bytes -- bytes of codes and scales for weights [N, K]. Errors as
 * mq_pack8's for N and K, and MQ_ERR_INVALID_ARG for a NULL result. */
mq_status mq_pack8_bytes(int64_t N, int64_t K, size_t* codes, size_t* scales);

/*
 * mq_pack8 -- fp16 weights as 8-bit rows in the order of mq_w8.
 *
 *   W_dev_fp16   [N, K] (nn.Linear layout [out, in]), rows w_stride elements
 *                apart, 2-byte aligned
 *   w            codes and scales to write, N and K
 *
 * A block with an Inf or NaN makes its output feature NaN for every token.
 * Errors: MQ_ERR_INVALID_ARG, MQ_ERR_UNSUPPORTED (K > 2^20, N > 2^24,
 * N * K8 >= 2^40), MQ_ERR_DEVICE.
 */
mq_status mq_pack8(const void* W_dev_fp16, int64_t w_stride, const mq_w8* w, void* hip_stream);

/*
 * mq_linear8 -- Y = X W^T of 8-bit rows and 8-bit weights.
 *
 *   codes_dev, scales_dev   [M, K8] and [M, K8 / 128] as mq_quantize8 writes
 *                them, rows codes_stride and scales_stride bytes apart; codes
 *                16-byte aligned with a stride that is a multiple of 16; codes
 *                past K are multiplied by zero weights: a NaN among them (as in a
 *                block that is NaN anyway) makes the token's outputs NaN
 *   M            tokens, >= 0 (0 enqueues nothing)
 *   w            from mq_pack8
 *   Y_dev_fp16   [M, N], rows y_stride elements apart (>= N), 2-byte aligned
 *   workspace_dev, workspace_bytes  at least mq_linear8_workspace bytes (0:
 *                NULL is accepted), 16-byte aligned; calls that overlap in time
 *                need their own
 *
 * Precision. The matrix instruction takes a block's 128 products in 16 groups
 * of 8 columns that follow each other. Products are exact, but of a group's the
 * part below 2^-13 of the power of two of its largest is cut off; the groups
 * join the sum in fp32, which is rounded once to fp16 (beyond its range: Inf).
 * With G the sum over all groups of the largest product's magnitude and P that
 * of all products', Y is off by at most
 *     2^-11 |Y| + 2^-25  +  7 2^-13 G  +  2^-19 (K8 / 128 + 1) P:
 * fp16's rounding, the cuts, and the fp32 sum (of that a mean of under 10^-5 P
 * was measured, at K = 2^20 and one sign). In sums of one sign all cuts go the same way: for
 * magnitudes over a range of 2^12 on both sides they take 8 10^-5 of Y, at worst,
 * where seven products of each group lie just under the cut, 8.5 10^-4 (half a
 * step of fp16 is 4.9 10^-4). Where products cancel, what is left may be smaller
 * than what was cut. Where the output tiles are too few to fill the GPU the sums
 * over K are split and joined in a fixed order. A token's outputs depend on its own row alone, but
 * their last bits may change with M, which chooses the split. Errors:
 * MQ_ERR_INVALID_ARG (also a workspace that is too small),
 * MQ_ERR_UNSUPPORTED (sizes as mq_pack8, M >= 2^24, codes_stride or
 * scales_stride > 2^22, or 2^24 workgroups of the plan or more: about
 * M N >= 2^39), MQ_ERR_DEVICE.
 */
mq_status mq_linear8(const void* codes_dev, int64_t codes_stride, const void* scales_dev, int64_t scales_stride,
                     int64_t M, const mq_w8* w, void* Y_dev_fp16, int64_t y_stride, void* workspace_dev,
                     size_t workspace_bytes, void* hip_stream);

/* mq_linear8_workspace -- bytes that mq_linear8 needs for M tokens and weights
 * of w's N and K (no pointer is read). */
mq_status mq_linear8_workspace(int64_t M, const mq_w8* w, size_t* bytes);

/*
 * mq_sample -- a token for each row of logits, from given random numbers.
 *
 * With l the row's logits, top its largest and t its temperature, token i has
 * the weight w_i = rint(2^40 exp((l_i - top) / t)), a whole number (computed
 * in fp64: a token less likely than 2^-41 of the likeliest has none). Tokens
 * are ordered by logit, the lower index first among equals. Kept is a token
 *   - that is among the first top_k (top_k <= 0: of all), and
 *   - with less than max(1, floor(top_p T)) of weight before it in that order,
 *     T the sum of the first top_k (top_p >= 1: of all; <= 0: the first alone),
 *   - with w_i >= min_p 2^40 (min_p <= 0: of all; more than 1 counts as 1).
 * With W the kept weights' sum the token drawn is the first, by index, whose
 * running sum of kept weights is more than floor(u W), and its log-probability
 * is ln(w / W). top_p and u count in steps of 2^-31. All sums are of
 * whole numbers, so no order of additions changes a result. t = 0 takes the
 * first largest logit (log-probability 0; no limit and no u is looked at).
 *
 * Logits may be -Inf (a token that may not be drawn). A row gets token -1 and
 * log-probability NaN where it has a NaN or +Inf logit or nothing but -Inf,
 * where t is negative, NaN or Inf, and, with t > 0, where top_p, min_p or u is
 * NaN. u below 0 counts as 0, from 1 on as 1 - 2^-31.
 */
typedef struct {
  const void* logits;          /* [rows, vocab] fp16 or fp32, rows `stride` elements apart, aligned to an element */
  int64_t rows;                /* >= 0 (0 enqueues nothing), <= 65535 */
  int64_t vocab;               /* 1 .. 2^22 */
  int64_t stride;              /* >= vocab, or 0: one row of logits for all */
  const float* temperature;    /* [rows], NULL: 1 */
  const int32_t* top_k;        /* [rows], NULL: all */
  const float* top_p;          /* [rows], NULL: all */
  const float* min_p;          /* [rows], NULL: all */
  const float* u;              /* [rows] uniform in [0, 1) */
  int32_t* token;              /* [rows] out */
  float* logprob;              /* [rows] out, or NULL */
  int32_t logits_fp32;         /* 0: fp16, 1: fp32 */
} mq_sample_args;

/* workspace as in mq_linear8. Errors: MQ_ERR_INVALID_ARG, MQ_ERR_UNSUPPORTED
 * (vocab > 2^22, rows > 65535), MQ_ERR_DEVICE. */
mq_status mq_sample(const mq_sample_args* args, void* workspace_dev, size_t workspace_bytes, void* hip_stream);

/* mq_sample_workspace -- bytes that mq_sample needs for these sizes (by rows,
 * vocab and logits_fp32; no pointer is read). */
mq_status mq_sample_workspace(const mq_sample_args* args, size_t* bytes);

#ifdef __cplusplus
}
#endif
#endif /* MOSAICQ_HEAD_H */
