// Host side of the block operators' C ABI (include/mosaicq_block.h): argument
// checks and dispatch to the kernels. No kernel code lives here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "block_internal.h"

#define MQ_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr int64_t k31 = int64_t(1) << 31;

mq_status from_hip(hipError_t e) {
  if (e == hipSuccess) return MQ_OK;
  if (e == hipErrorOutOfMemory) return MQ_ERR_OUT_OF_MEMORY;
  return MQ_ERR_DEVICE;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A rope plan for heads of head_dim elements.
mq_status check_plan(const mq_rope_plan* r, int64_t head_dim) {
  if (!r->table || !aligned(r->table, 8) || r->positions <= 0) return MQ_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > head_dim) return MQ_ERR_INVALID_ARG;
  if (r->layout != MQ_ROPE_HALF && r->layout != MQ_ROPE_INTERLEAVED) return MQ_ERR_INVALID_ARG;
  return MQ_OK;
}

mq::RopeView view(const mq_rope_plan* r) {
  if (!r) return {nullptr, 0, 0, 0};
  return {reinterpret_cast<const float2*>(r->table), r->positions, r->rot_dim, r->layout == MQ_ROPE_INTERLEAVED};
}

mq_status check_cache_sizes(const mq_kv_cache* c) {
  if (!c || c->num_blocks <= 0 || c->num_slots <= 0 || c->kv_heads <= 0 || c->kv_heads > 1024)
    return MQ_ERR_INVALID_ARG;
  if (c->format != MQ_KV_INT8 && c->format != MQ_KV_E4M3) return MQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MQ_ERR_UNSUPPORTED;
  if (c->num_slots >= k31 || c->num_blocks >= k31) return MQ_ERR_UNSUPPORTED;
  return MQ_OK;
}

mq_status check_cache(const mq_kv_cache* c) {
  const mq_status st = check_cache_sizes(c);
  if (st != MQ_OK) return st;
  for (const void* p : {c->k_codes, c->v_codes, c->k_tail, c->v_tail})
    if (!p || !aligned(p, 16)) return MQ_ERR_INVALID_ARG;
  for (const float* p : {c->k_scale, c->v_scale})
    if (!p || !aligned(p, 4)) return MQ_ERR_INVALID_ARG;
  return MQ_OK;
}

mq_status check_batch_sizes(const mq_kv_batch* b) {
  if (!b || b->seqs < 0 || b->seqs > 65535 || b->tokens < 0 || b->max_new <= 0 || b->max_len <= 0)
    return MQ_ERR_INVALID_ARG;
  if (b->tokens >= k31 || b->max_new >= k31 || b->max_len >= k31) return MQ_ERR_UNSUPPORTED;
  return MQ_OK;
}

mq_status check_batch(const mq_kv_batch* b) {
  const mq_status st = check_batch_sizes(b);
  if (st != MQ_OK) return st;
  if (b->table_width <= 0) return MQ_ERR_INVALID_ARG;
  if (b->table_width >= k31) return MQ_ERR_UNSUPPORTED;
  for (const int32_t* p : {b->cu_q, b->kv_len, b->block_table})
    if (!p || !aligned(p, 4)) return MQ_ERR_INVALID_ARG;
  return b->slots && !aligned(b->slots, 4) ? MQ_ERR_INVALID_ARG : MQ_OK;
}

mq::KvView view(const mq_kv_cache* c) {
  return {static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes), c->k_scale, c->v_scale,
          static_cast<_Float16*>(c->k_tail), static_cast<_Float16*>(c->v_tail), c->num_blocks, (int)c->num_slots,
          c->kv_heads};
}

mq::BatchView view(const mq_kv_batch* b) {
  return {b->cu_q, b->kv_len, b->block_table, b->slots, (int)b->seqs, (int)b->tokens, (int)b->table_width,
          (int)b->max_new, (int)b->max_len};
}

// fp16 rows of `width` elements.
bool bad_rows(const void* p, int64_t stride, int64_t width, size_t align = 2) {
  return !p || !aligned(p, align) || stride < width || (stride * 2) % (int64_t)align != 0;
}

}  // namespace

MQ_API mq_status mq_rope_table(const mq_rope_spec* spec, int64_t positions, float* table_dev_f32, void* hip_stream) {
  if (!spec || !table_dev_f32 || !aligned(table_dev_f32, 8) || positions <= 0) return MQ_ERR_INVALID_ARG;
  const int32_t rot = spec->rot_dim;
  if (rot < 2 || rot % 2 != 0 || rot > 1024) return MQ_ERR_INVALID_ARG;
  if (spec->scaling < MQ_ROPE_NONE || spec->scaling > MQ_ROPE_PARTS) return MQ_ERR_INVALID_ARG;
  if (!(spec->theta > 1.0) || !std::isfinite(spec->theta)) return MQ_ERR_INVALID_ARG;
  if (spec->scaling != MQ_ROPE_NONE && (!(spec->factor >= 1.0) || !std::isfinite(spec->factor)))
    return MQ_ERR_INVALID_ARG;
  const bool parts = spec->scaling == MQ_ROPE_PARTS;
  if (parts && (!(spec->original > 0.0) || !std::isfinite(spec->original) || !(spec->turns_slow > 0.0) ||
                !(spec->turns_fast > spec->turns_slow) || !std::isfinite(spec->turns_fast)))
    return MQ_ERR_INVALID_ARG;
  if (positions >= k31 / rot) return MQ_ERR_UNSUPPORTED;

  double theta = spec->theta, mag = 1.0, lo = 0.0, hi = 1.0;
  if (spec->scaling == MQ_ROPE_BASE) theta *= std::pow(spec->factor, rot / (double)std::max(1, rot - 2));
  if (parts) {
    const auto pair_of = [&](double turns) {
      return rot * std::log(spec->original / (turns * 2.0 * M_PI)) / (2.0 * std::log(spec->theta));
    };
    lo = std::max(0.0, std::floor(pair_of(spec->turns_fast)));
    hi = std::min(rot - 1.0, std::ceil(pair_of(spec->turns_slow)));
    mag = 0.1 * std::log(spec->factor) + 1.0;
  }
  double f[512];
  for (int i = 0; i < rot / 2; ++i) {
    f[i] = std::pow(theta, -2.0 * i / rot);
    if (spec->scaling == MQ_ROPE_LINEAR) f[i] /= spec->factor;
    if (parts) {
      const double r = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
      f[i] = f[i] * (1.0 - r) + f[i] / spec->factor * r;
    }
  }
  return from_hip(mq::launch_rope_table(f, rot / 2, mag, positions, reinterpret_cast<float2*>(table_dev_f32),
                                        static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_rope(const void* X_dev_fp16, int64_t tokens, int32_t heads, int32_t head_dim,
                         int64_t x_token_stride, int64_t x_head_stride, const int32_t* pos_dev_i32,
                         const mq_rope_plan* rope, int32_t inverse, void* Y_dev_fp16, int64_t y_token_stride,
                         int64_t y_head_stride, void* hip_stream) {
  if (!X_dev_fp16 || !pos_dev_i32 || !rope || !Y_dev_fp16 || tokens < 0 || heads <= 0 || head_dim < 2)
    return MQ_ERR_INVALID_ARG;
  if (!aligned(X_dev_fp16, 2) || !aligned(Y_dev_fp16, 2) || !aligned(pos_dev_i32, 4)) return MQ_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return MQ_ERR_INVALID_ARG;
  for (const int64_t t : {x_token_stride, x_head_stride, y_token_stride, y_head_stride})
    if (t < 0) return MQ_ERR_INVALID_ARG;
  // outputs of different tokens or heads must not fall on each other
  if ((heads > 1 && y_head_stride < head_dim) || (tokens > 1 && y_token_stride < head_dim)) return MQ_ERR_INVALID_ARG;
  const mq_status st = check_plan(rope, head_dim);
  if (st != MQ_OK) return st;
  if (tokens >= k31 || (int64_t)heads * head_dim >= k31) return MQ_ERR_UNSUPPORTED;
  return from_hip(mq::launch_rope(static_cast<const _Float16*>(X_dev_fp16), tokens, heads, head_dim, x_token_stride,
                                  x_head_stride, pos_dev_i32, view(rope), inverse,
                                  static_cast<_Float16*>(Y_dev_fp16), y_token_stride, y_head_stride,
                                  static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_kv_append(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q_dev_fp16,
                              int32_t q_heads, int64_t q_stride, const void* k_dev_fp16, int64_t k_stride,
                              const void* v_dev_fp16, int64_t v_stride, const mq_rope_plan* rope,
                              void* q_out_dev_fp16, int64_t q_out_stride, void* hip_stream) {
  mq_status st = check_cache(cache);
  if (st == MQ_OK) st = check_batch(batch);
  if (st != MQ_OK) return st;
  const int64_t D = cache->head_dim, kw = cache->kv_heads * D;
  if (bad_rows(k_dev_fp16, k_stride, kw) || bad_rows(v_dev_fp16, v_stride, kw)) return MQ_ERR_INVALID_ARG;
  const bool queries = rope && q_dev_fp16;
  if (rope) {
    st = check_plan(rope, D);
    if (st != MQ_OK) return st;
  }
  if (queries) {
    if (q_heads <= 0 || q_heads >= (1 << 20)) return MQ_ERR_INVALID_ARG;
    if (bad_rows(q_dev_fp16, q_stride, q_heads * D) || bad_rows(q_out_dev_fp16, q_out_stride, q_heads * D))
      return MQ_ERR_INVALID_ARG;
  }
  bool too_large = false;
  const hipError_t e = mq::launch_kv_append(
      view(cache), cache->head_dim, cache->format, view(batch),
      {queries ? static_cast<const _Float16*>(q_dev_fp16) : nullptr, q_stride}, q_heads,
      {static_cast<const _Float16*>(k_dev_fp16), k_stride}, {static_cast<const _Float16*>(v_dev_fp16), v_stride},
      view(rope), {static_cast<_Float16*>(q_out_dev_fp16), q_out_stride}, &too_large,
      static_cast<hipStream_t>(hip_stream));
  return too_large ? MQ_ERR_UNSUPPORTED : from_hip(e);
}

namespace {

// What both attention entry points need: sizes, heads, and the plan.
mq_status attention_plan(const mq_kv_cache* cache, const mq_kv_batch* batch, int32_t q_heads, mq::AttnPlan* plan) {
  mq_status st = check_cache_sizes(cache);
  if (st == MQ_OK) st = check_batch_sizes(batch);
  if (st != MQ_OK) return st;
  if (q_heads <= 0 || q_heads % cache->kv_heads != 0) return MQ_ERR_INVALID_ARG;
  if (q_heads / cache->kv_heads > 64) return MQ_ERR_UNSUPPORTED;
  *plan = mq::plan_attention(cache->kv_heads, q_heads, cache->head_dim, batch->seqs, batch->tokens, batch->max_new,
                             batch->max_len);
  return mq::launchable(plan->groups, plan->threads) && mq::launchable(plan->joins, 256) ? MQ_OK : MQ_ERR_UNSUPPORTED;
}

}  // namespace

MQ_API mq_status mq_kv_attention_workspace(const mq_kv_cache* cache, const mq_kv_batch* batch, int32_t q_heads,
                                           size_t* bytes) {
  if (!bytes) return MQ_ERR_INVALID_ARG;
  mq::AttnPlan plan;
  const mq_status st = attention_plan(cache, batch, q_heads, &plan);
  if (st == MQ_OK) *bytes = plan.bytes;
  return st;
}

MQ_API mq_status mq_kv_attention(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q_dev_fp16,
                                 int32_t q_heads, int64_t q_stride, int32_t causal, float scale, void* out_dev_fp16,
                                 int64_t out_stride, void* workspace_dev, size_t workspace_bytes, void* hip_stream) {
  mq_status st = check_cache(cache);
  if (st == MQ_OK) st = check_batch(batch);
  if (st != MQ_OK) return st;
  mq::AttnPlan plan;
  st = attention_plan(cache, batch, q_heads, &plan);
  if (st != MQ_OK) return st;
  const int64_t width = (int64_t)q_heads * cache->head_dim;
  if (bad_rows(q_dev_fp16, q_stride, width, 16) || bad_rows(out_dev_fp16, out_stride, width, 8))
    return MQ_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || (causal != 0 && causal != 1)) return MQ_ERR_INVALID_ARG;
  if (plan.bytes > 0 && (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < plan.bytes))
    return MQ_ERR_INVALID_ARG;
  return from_hip(mq::launch_kv_attention(view(cache), cache->head_dim, cache->format, view(batch),
                                          {static_cast<const _Float16*>(q_dev_fp16), q_stride}, q_heads, causal, scale,
                                          {static_cast<_Float16*>(out_dev_fp16), out_stride}, workspace_dev, plan,
                                          static_cast<hipStream_t>(hip_stream)));
}

MQ_API mq_status mq_norm_residual(const mq_norm_args* args, void* hip_stream) {
  if (!args) return MQ_ERR_INVALID_ARG;
  const mq_norm_args& a = *args;
  if (a.tokens < 0 || a.width <= 0 || !a.r || (!a.y && !a.w_pre)) return MQ_ERR_INVALID_ARG;
  if (a.residual_fp32 != 0 && a.residual_fp32 != 1) return MQ_ERR_INVALID_ARG;
  const size_t rs = a.residual_fp32 ? 4 : 2;
  if (!aligned(a.r, rs) || a.r_stride < a.width) return MQ_ERR_INVALID_ARG;
  if (a.y) {
    if (bad_rows(a.y, a.y_stride, a.width) || !a.r_out || !aligned(a.r_out, rs) || a.r_out_stride < a.width)
      return MQ_ERR_INVALID_ARG;
    if (a.gate && (!aligned(a.gate, 2) || (a.gate_stride != 0 && a.gate_stride < a.width))) return MQ_ERR_INVALID_ARG;
    if (!std::isfinite(a.alpha) || !std::isfinite(a.beta)) return MQ_ERR_INVALID_ARG;
  }
  if (!aligned(a.w_post, 2) || !aligned(a.w_pre, 2)) return MQ_ERR_INVALID_ARG;
  if (a.w_pre && bad_rows(a.h_out, a.h_stride, a.width)) return MQ_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f) || !std::isfinite(a.eps) || !std::isfinite(a.weight_offset)) return MQ_ERR_INVALID_ARG;
  if (a.width > 65536 || a.tokens >= k31) return MQ_ERR_UNSUPPORTED;
  return from_hip(mq::launch_norm_residual(a, static_cast<hipStream_t>(hip_stream)));
}
