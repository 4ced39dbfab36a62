// C ABI of the rotary positions, the 8-bit key/value cache and the attention
// over it: argument checks and dispatch.  Nothing is enqueued unless every
// argument that the host can see is valid.
#include <cmath>

#include "../../include/mq.h"
#include "mq_internal.h"

namespace {

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

constexpr int64_t kMaxRowEntries = (int64_t)1 << 20;  // heads * dim
constexpr int64_t kMaxNew = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

mq_status check_cache(const mq_kv_cache* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return MQ_ERR_NULL;
  if (c->format != MQ_KV_INT8 && c->format != MQ_KV_E4M3) return MQ_ERR_PRECISION;
  if (c->pages < 1 || c->pages > 0x7fffffff || c->heads < 1 || c->heads > 4096) return MQ_ERR_SHAPE;
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128) return MQ_ERR_SHAPE;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return MQ_ERR_SHAPE;
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) ||
      misaligned(c->v_scale, 4))
    return MQ_ERR_ALIGN;
  return MQ_OK;
}

mq_status check_batch(const mq_kv_batch* b, const mq_kv_cache* c) {
  if (!b || !b->q_start || !b->kv_len || !b->page_table) return MQ_ERR_NULL;
  if (b->rows < 0 || b->rows > 0x7fffffff || b->seqs < 1 || b->seqs > 65535) return MQ_ERR_SHAPE;
  if (b->table_pages < 1 || (int64_t)b->table_pages * c->block > (int64_t)1 << 30) return MQ_ERR_SHAPE;
  if (b->max_new < 1 || b->max_new > kMaxNew) return MQ_ERR_SHAPE;
  if (misaligned(b->q_start, 4) || misaligned(b->kv_len, 4) || misaligned(b->page_table, 4))
    return MQ_ERR_ALIGN;
  return MQ_OK;
}

mq_status check_rope(const mq_rope_spec* r, int64_t dim) {
  if (!r || !r->freq) return MQ_ERR_NULL;
  if (r->rot < 8 || r->rot % 8 != 0 || r->rot > dim) return MQ_ERR_SHAPE;
  if ((r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->factor))
    return MQ_ERR_PRECISION;
  if (misaligned(r->freq, 8)) return MQ_ERR_ALIGN;
  return MQ_OK;
}

// rows of `entries` consecutive entries every `stride`
mq_status check_strided(const void* p, int64_t stride, int64_t entries) {
  if (stride < entries || stride > kMaxStride) return MQ_ERR_SHAPE;
  if (stride % 8 != 0 || misaligned(p, 16)) return MQ_ERR_ALIGN;
  return MQ_OK;
}

mq::KvCache cache_of(const mq_kv_cache* c) {
  return mq::KvCache{c->k, c->v, c->k_scale, c->v_scale, (int)c->pages, c->heads, c->block, c->dim,
                     c->format == MQ_KV_E4M3};
}
mq::KvBatch batch_of(const mq_kv_batch* b) {
  return mq::KvBatch{b->q_start, b->kv_len, b->page_table, b->rows, b->seqs, b->table_pages,
                     b->max_new};
}
mq::RopeSpec rope_of(const mq_rope_spec* r) {
  if (!r) return mq::RopeSpec{nullptr, 1.0, 0, 0};
  return mq::RopeSpec{r->freq, r->factor, r->rot, r->interleaved};
}

mq_status done(hipError_t e) { return e == hipSuccess ? MQ_OK : mq::record_hip_error(e); }

mq_status check_attend(const mq_kv_cache* c, const mq_kv_batch* b, int64_t q_heads,
                       int64_t window) {
  mq_status s = check_cache(c);
  if (s != MQ_OK) return s;
  s = check_batch(b, c);
  if (s != MQ_OK) return s;
  if (q_heads < 1 || q_heads > kMaxRowEntries / c->dim || q_heads % c->heads != 0 ||
      q_heads / c->heads > 1024)
    return MQ_ERR_SHAPE;
  if ((int64_t)b->max_new * q_heads > (int64_t)1 << 24) return MQ_ERR_SHAPE;
  if (b->rows * q_heads > (int64_t)1 << 25) return MQ_ERR_SHAPE;  // 64 threads each, one grid
  if (window < 0) return MQ_ERR_SHAPE;
  return MQ_OK;
}

mq::AttendArgs attend_args(const mq_kv_cache* c, const mq_kv_batch* b, int64_t q_heads,
                           int64_t window) {
  mq::AttendArgs a{};
  a.cache = cache_of(c);
  a.batch = batch_of(b);
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / c->heads);
  a.group_mul = (((uint64_t)1 << 36) + a.group - 1) / a.group;
  a.window = window < (int64_t)1 << 31 ? window : (int64_t)1 << 31;  // no position is beyond
  return a;
}

}  // namespace

namespace mq {

mq_status append_check(const mq_kv_cache* cache, const mq_kv_batch* batch,
                       const mq_rope_spec* rope, const void* k, const void* v, int64_t kv_stride,
                       const void* q, int64_t q_stride, int64_t q_heads, int x_type,
                       const uint16_t* q_out) {
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return MQ_ERR_NULL;
  mq_status s = check_cache(cache);
  if (s != MQ_OK) return s;
  s = check_batch(batch, cache);
  if (s != MQ_OK) return s;
  if (x_type != MQ_BF16 && x_type != MQ_F32) return MQ_ERR_PRECISION;
  const int64_t dim = cache->dim;
  if (rope && (s = check_rope(rope, dim)) != MQ_OK) return s;
  if (cache->heads > kMaxRowEntries / dim) return MQ_ERR_SHAPE;
  if ((s = check_strided(k, kv_stride, cache->heads * dim)) != MQ_OK) return s;
  if ((s = check_strided(v, kv_stride, cache->heads * dim)) != MQ_OK) return s;
  if (q) {
    if (q_heads < 1 || q_heads > kMaxRowEntries / dim) return MQ_ERR_SHAPE;
    if ((s = check_strided(q, q_stride, q_heads * dim)) != MQ_OK) return s;
    if (misaligned(q_out, 16)) return MQ_ERR_ALIGN;
  }
  return MQ_OK;
}

mq_status attend_check(const mq_kv_cache* cache, const mq_kv_batch* batch, const uint16_t* q,
                       int64_t q_stride, int64_t q_heads, float scale, float softcap,
                       int64_t window, int causal, const uint16_t* out, const float* lse) {
  if (!q || !out) return MQ_ERR_NULL;
  mq_status s = check_attend(cache, batch, q_heads, window);
  if (s != MQ_OK) return s;
  if (!std::isfinite(scale) || !(softcap >= 0.f && softcap <= 1e6f) ||
      (softcap > 0.f && softcap < 1e-6f) || (causal != 0 && causal != 1))
    return MQ_ERR_PRECISION;
  if (window > 0 && !causal) return MQ_ERR_SHAPE;
  if ((s = check_strided(q, q_stride, q_heads * cache->dim)) != MQ_OK) return s;
  if (misaligned(out, 16) || misaligned(lse, 4)) return MQ_ERR_ALIGN;
  return MQ_OK;
}

}  // namespace mq

extern "C" {

mq_status mq_rope(const mq_rope_spec* rope, const int32_t* positions, const void* x, int x_type,
                  int64_t x_stride, int64_t rows, int64_t heads, int64_t dim, uint16_t* out,
                  int64_t out_stride, void* stream) {
  if (!rope || !rope->freq || !positions || !x || !out) return MQ_ERR_NULL;
  if (x_type != MQ_BF16 && x_type != MQ_F32) return MQ_ERR_PRECISION;
  if (rows < 0 || rows > kMaxNew || heads < 1 || dim < 8 || dim > 1024 || dim % 8 != 0 ||
      heads > kMaxRowEntries / dim)
    return MQ_ERR_SHAPE;
  mq_status s = check_rope(rope, dim);
  if (s != MQ_OK) return s;
  if ((s = check_strided(x, x_stride, heads * dim)) != MQ_OK) return s;
  if ((s = check_strided(out, out_stride, heads * dim)) != MQ_OK) return s;
  if (misaligned(positions, 4)) return MQ_ERR_ALIGN;
  if (x == out && (x_type != MQ_BF16 || x_stride != out_stride)) return MQ_ERR_SHAPE;
  s = mq::device_check();
  if (s != MQ_OK) return s;
  return done(mq::launch_rope(rope_of(rope), positions, x, x_type == MQ_F32, x_stride, rows,
                              (int)heads, (int)dim, out, out_stride, (hipStream_t)stream));
}

mq_status mq_cache_append(const mq_kv_cache* cache, const mq_kv_batch* batch,
                          const mq_rope_spec* rope, const void* k, const void* v,
                          int64_t kv_stride, const void* q, int64_t q_stride, int64_t q_heads,
                          int x_type, uint16_t* q_out, void* stream) {
  mq_status s = mq::append_check(cache, batch, rope, k, v, kv_stride, q, q_stride, q_heads, x_type,
                                 q_out);
  if (s != MQ_OK) return s;
  s = mq::device_check();
  if (s != MQ_OK) return s;
  return done(mq::launch_cache_append(cache_of(cache), batch_of(batch), rope_of(rope), k, v,
                                      kv_stride, q, q_stride, q ? (int)q_heads : 0,
                                      x_type == MQ_F32, q_out, (hipStream_t)stream));
}

mq_status mq_cache_read(const mq_kv_cache* cache, const mq_kv_batch* batch, void* k_out,
                        void* v_out, int out_type, void* stream) {
  if (!k_out && !v_out) return MQ_ERR_NULL;
  mq_status s = check_cache(cache);
  if (s != MQ_OK) return s;
  s = check_batch(batch, cache);
  if (s != MQ_OK) return s;
  if (out_type != MQ_BF16 && out_type != MQ_F32) return MQ_ERR_PRECISION;
  if (misaligned(k_out, 16) || misaligned(v_out, 16)) return MQ_ERR_ALIGN;
  s = mq::device_check();
  if (s != MQ_OK) return s;
  return done(mq::launch_cache_read(cache_of(cache), batch_of(batch), k_out, v_out,
                                    out_type == MQ_F32, (hipStream_t)stream));
}

size_t mq_cache_attend_workspace_bytes(const mq_kv_cache* cache, const mq_kv_batch* batch,
                                       int64_t q_heads, int64_t window) {
  if (check_attend(cache, batch, q_heads, window) != MQ_OK) return 0;
  return mq::attend_plan(attend_args(cache, batch, q_heads, window), nullptr).bytes;
}

mq_status mq_cache_attend(const mq_kv_cache* cache, const mq_kv_batch* batch, const uint16_t* q,
                          int64_t q_stride, int64_t q_heads, float scale, float softcap,
                          int64_t window, int causal, uint16_t* out, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  mq_status s = mq::attend_check(cache, batch, q, q_stride, q_heads, scale, softcap, window, causal,
                                 out, lse);
  if (s != MQ_OK) return s;
  mq::AttendArgs a = attend_args(cache, batch, q_heads, window);
  const mq::AttendPlan plan = mq::attend_plan(a, workspace);
  const size_t need = plan.bytes;
  if (need > 0 && (!workspace || workspace_bytes < need)) return MQ_ERR_WORKSPACE;
  if (need > 0 && misaligned(workspace, 256)) return MQ_ERR_ALIGN;
  s = mq::device_check();
  if (s != MQ_OK) return s;
  a.q = q;
  a.q_stride = q_stride;
  a.scale = scale;
  a.softcap = softcap;
  a.causal = causal;
  a.out = out;
  a.lse = lse;
  return done(mq::launch_attend(a, plan, (hipStream_t)stream));
}

}  // extern "C"
