// CPU build of the packer's exact integer arithmetic (quant_exact.h) and of the
// rules by which the head's operators choose their kernels (head_plan.h),
// exported for tests that run without a GPU. The libraries compile the same
// headers.
#include <cstdint>

#include "head_plan.h"
#include "quant_exact.h"

#define HC_API extern "C" __attribute__((visibility("default")))

HC_API int64_t mqh_fp16_units(uint32_t h) { return mq::fp16_units(h); }
HC_API uint32_t mqh_fp16_div7(uint64_t A, uint64_t* S) { return mq::fp16_div7(A, S); }
HC_API uint32_t mqh_fp16_round_units(uint64_t V, uint64_t* R) { return mq::fp16_round_units(V, R); }
HC_API uint32_t mqh_fp32_div7(uint64_t Mx, uint64_t* m, int* Q) { return mq::fp32_div7(Mx, m, Q); }
HC_API int mqh_quant7(int64_t a, uint64_t S) { return mq::quant7(a, S); }
HC_API int mqh_quant7_scaled(int64_t e, uint64_t m, int Q) { return mq::quant7_scaled(e, m, Q); }
HC_API uint64_t mqh_err_key(uint64_t abs_e) { return mq::err_key(abs_e); }
HC_API uint32_t mqh_fp16_div7_h(uint32_t h) { return mq::fp16_div7_h(h); }
HC_API int mqh_quant7_f(float x, float s) { return mq::quant7_f(x, s); }

// nt, r, waves, tb, splits, per of the plan; its workspace's bytes
HC_API int64_t mqh_linear8_plan(int64_t M, int64_t N, int64_t K, int* plan) {
  const mq::Linear8Plan p = mq::plan_linear8(M, N, K);
  const int fields[] = {p.nt, p.r, p.waves, p.tb, p.splits, p.per};
  for (int i = 0; i < 6; ++i) plan[i] = fields[i];
  return (int64_t)p.bytes;
}
// Whether a workgroup takes a row; else a row's workgroups and the tokens of a segment.
HC_API int mqh_sample_by_rows(int64_t rows, int64_t vocab, int* splits, int* span) {
  mq::split(rows, vocab, splits, span);
  return mq::by_rows(rows, vocab);
}
