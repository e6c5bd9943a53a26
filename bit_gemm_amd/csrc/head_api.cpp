// Host side of the head's C ABI (include/mosaicq_head.h): argument checks and
// dispatch to the kernels. No kernel code lives here.
#include <hip/hip_runtime.h>

#include "head_internal.h"

#define MQ_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t k31 = int64_t(1) << 31;
constexpr int64_t kMostK = int64_t(1) << 20;
constexpr int64_t kMostRows = int64_t(1) << 24;
// The tiled kernel addresses a workgroup's 128 token rows by offsets under 2^30.
constexpr int64_t kMostStride = int64_t(1) << 22;

mq_status from_hip(hipError_t e) {
  if (e == hipSuccess) return MQ_OK;
  if (e == hipErrorOutOfMemory) return MQ_ERR_OUT_OF_MEMORY;
  return MQ_ERR_DEVICE;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t blocks(int64_t K) { return (K + 127) / 128; }

// Rows of 8 bits: addresses and strides.
bool bad_rows8(const void* codes, int64_t stride, const void* scales, int64_t sstride, int64_t K) {
  return !codes || !aligned(codes, 16) || stride < 128 * blocks(K) || stride % 16 != 0 || !scales || sstride < blocks(K);
}

mq_status check_sizes(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0) return MQ_ERR_INVALID_ARG;
  if (K > kMostK || N > kMostRows || N * 128 * blocks(K) >= (int64_t(1) << 40)) return MQ_ERR_UNSUPPORTED;
  return MQ_OK;
}

mq_status check_w8(const mq_w8* w) {
  if (!w || !w->codes || !aligned(w->codes, 16) || !w->scales || !aligned(w->scales, 4)) return MQ_ERR_INVALID_ARG;
  return check_sizes(w->N, w->K);
}

mq::W8 view(const mq_w8* w) {
  const int64_t Kt = blocks(w->K);
  return {static_cast<const uint8_t*>(w->codes), static_cast<const uint8_t*>(w->scales), w->N, w->K,
          (int)((w->N + 15) / 16), (int)Kt, (int)((Kt + 3) / 4)};
}

// The plan of a product, where it can be run.
mq_status linear_plan(int64_t M, const mq_w8* w, mq::Linear8Plan* plan) {
  if (!w || M < 0) return MQ_ERR_INVALID_ARG;
  const mq_status st = check_sizes(w->N, w->K);
  if (st != MQ_OK) return st;
  if (M >= kMostRows) return MQ_ERR_UNSUPPORTED;
  *plan = mq::plan_linear8(M, w->N, w->K);
  if (plan->groups >= kMostRows) return MQ_ERR_UNSUPPORTED;   // a launch takes fewer than 2^32 threads
  return MQ_OK;
}

mq_status check_sample_sizes(const mq_sample_args* a) {
  if (!a || a->rows < 0 || a->vocab <= 0 || (a->logits_fp32 != 0 && a->logits_fp32 != 1)) return MQ_ERR_INVALID_ARG;
  if (a->rows > 65535 || a->vocab > (int64_t(1) << 22)) return MQ_ERR_UNSUPPORTED;
  return MQ_OK;
}

}  // namespace

MQ_API mq_status mq_quantize8(const void* X_dev_fp16, int64_t M, int64_t K, int64_t x_stride, void* codes_dev,
                              int64_t codes_stride, void* scales_dev, int64_t scales_stride, void* hip_stream) {
  if (M < 0 || K <= 0 || !X_dev_fp16 || !aligned(X_dev_fp16, 2) || x_stride < K) return MQ_ERR_INVALID_ARG;
  if (K > kMostK || M >= k31 || M * 128 * blocks(K) >= (int64_t(1) << 42)) return MQ_ERR_UNSUPPORTED;
  if (bad_rows8(codes_dev, codes_stride, scales_dev, scales_stride, K)) return MQ_ERR_INVALID_ARG;
  return from_hip(mq::launch_quantize8(static_cast<const _Float16*>(X_dev_fp16), M, K, x_stride,
                                       static_cast<uint8_t*>(codes_dev), codes_stride,
                                       static_cast<uint8_t*>(scales_dev), scales_stride,
                                       static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_pack8_bytes(int64_t N, int64_t K, size_t* codes, size_t* scales) {
  if (!codes || !scales) return MQ_ERR_INVALID_ARG;
  const mq_status st = check_sizes(N, K);
  if (st != MQ_OK) return st;
  const size_t Nb = (size_t)((N + 15) / 16), Kt = (size_t)blocks(K);
  *codes = Nb * Kt * 2048;
  *scales = Nb * ((Kt + 3) / 4) * 64;
  return MQ_OK;
}

MQ_API mq_status mq_pack8(const void* W_dev_fp16, int64_t w_stride, const mq_w8* w, void* hip_stream) {
  const mq_status st = check_w8(w);
  if (st != MQ_OK) return st;
  if (!W_dev_fp16 || !aligned(W_dev_fp16, 2) || w_stride < w->K) return MQ_ERR_INVALID_ARG;
  return from_hip(mq::launch_pack8(static_cast<const _Float16*>(W_dev_fp16), w_stride, view(w),
                                   static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_linear8_workspace(int64_t M, const mq_w8* w, size_t* bytes) {
  if (!bytes) return MQ_ERR_INVALID_ARG;
  mq::Linear8Plan plan;
  const mq_status st = linear_plan(M, w, &plan);
  if (st == MQ_OK) *bytes = plan.bytes;
  return st;
}

MQ_API mq_status mq_linear8(const void* codes_dev, int64_t codes_stride, const void* scales_dev,
                            int64_t scales_stride, int64_t M, const mq_w8* w, void* Y_dev_fp16, int64_t y_stride,
                            void* workspace_dev, size_t workspace_bytes, void* hip_stream) {
  mq_status st = check_w8(w);
  if (st != MQ_OK) return st;
  mq::Linear8Plan plan;
  st = linear_plan(M, w, &plan);
  if (st != MQ_OK) return st;
  if (bad_rows8(codes_dev, codes_stride, scales_dev, scales_stride, w->K)) return MQ_ERR_INVALID_ARG;
  if (codes_stride > kMostStride || scales_stride > kMostStride) return MQ_ERR_UNSUPPORTED;
  if (!Y_dev_fp16 || !aligned(Y_dev_fp16, 2) || y_stride < w->N) return MQ_ERR_INVALID_ARG;
  if (plan.bytes > 0 && (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < plan.bytes))
    return MQ_ERR_INVALID_ARG;
  if (M == 0) return MQ_OK;
  return from_hip(mq::launch_linear8({static_cast<const uint8_t*>(codes_dev), static_cast<const uint8_t*>(scales_dev),
                                      codes_stride, scales_stride}, M, view(w), static_cast<_Float16*>(Y_dev_fp16),
                                     y_stride, workspace_dev, plan, static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_sample_workspace(const mq_sample_args* args, size_t* bytes) {
  if (!bytes) return MQ_ERR_INVALID_ARG;
  const mq_status st = check_sample_sizes(args);
  if (st == MQ_OK) *bytes = mq::sample_workspace(args->rows, args->vocab, args->logits_fp32);
  return st;
}

MQ_API mq_status mq_sample(const mq_sample_args* args, void* workspace_dev, size_t workspace_bytes, void* hip_stream) {
  const mq_status st = check_sample_sizes(args);
  if (st != MQ_OK) return st;
  const mq_sample_args& a = *args;
  if (!a.logits || !aligned(a.logits, a.logits_fp32 ? 4 : 2) || (a.stride != 0 && a.stride < a.vocab)) return MQ_ERR_INVALID_ARG;
  if (!a.u || !a.token) return MQ_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a.temperature, (const void*)a.top_k, (const void*)a.top_p, (const void*)a.min_p,
                        (const void*)a.u, (const void*)a.token, (const void*)a.logprob})
    if (!aligned(p, 4)) return MQ_ERR_INVALID_ARG;
  const size_t need = mq::sample_workspace(a.rows, a.vocab, a.logits_fp32);
  if (need > 0 && (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < need)) return MQ_ERR_INVALID_ARG;
  if (a.rows == 0) return MQ_OK;
  return from_hip(mq::launch_sample(a, workspace_dev, static_cast<hipStream_t>(hip_stream)));
}
