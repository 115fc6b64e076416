// Host side of the append entry points (include/verify_attn.h): argument
// validation and the launch.
#include <climits>
#include <cmath>
#include <cstring>

#include "va_append.h"
#include "va_host_impl.h"

namespace va_host_impl {
using namespace va;

// The metadata every append call takes: block table, prefix sums, lengths.
va_status check_batch(const va_tensor* bt, const va_tensor* cu, const va_tensor* su) {
  if (!dims_ok(bt, 2) || !dims_ok(cu, 1) || !dims_ok(su, 1)) return VA_ERR_SHAPE;
  if (bt->dtype != VA_INT32 || cu->dtype != VA_INT32 || su->dtype != VA_INT32) return VA_ERR_DTYPE;
  const int64_t B = su->shape[0];
  if (cu->shape[0] != B + 1 || bt->shape[0] != B) return VA_ERR_SHAPE;
  if (B > INT32_MAX / 4 || bt->shape[1] > INT32_MAX / kPageSize) return VA_ERR_UNSUPPORTED;
  if (cu->stride[0] != 1 || su->stride[0] != 1) return VA_ERR_LAYOUT;
  if (!cu->data || (B > 0 && !su->data) || (numel(bt) > 0 && !bt->data)) return VA_ERR_NULL;
  return VA_OK;
}

// Rows that are read or written in 16-byte pieces: present and aligned.
va_status check_rows(const va_tensor* t) {
  if (!rows_16b(t)) return VA_ERR_LAYOUT;
  if (numel(t) > 0 && !t->data) return VA_ERR_NULL;
  if (t->data && !aligned16(t->data)) return VA_ERR_LAYOUT;
  return VA_OK;
}

// Whether the elements of a tensor that is written have places of their own:
// runs of `width` elements over its first `dims` dimensions, whose strides are
// nested in some order (each at least what the ones inside it span).
bool places_distinct(const va_tensor* t, int dims, int64_t width) {
  int order[4], n = 0;
  for (int i = 0; i < dims; ++i) {
    if (t->shape[i] <= 1) continue;
    int j = n++;
    for (; j > 0 && t->stride[order[j - 1]] > t->stride[i]; --j) order[j] = order[j - 1];
    order[j] = i;
  }
  int64_t span = width;
  for (int j = 0; j < n; ++j) {
    const int64_t stride = t->stride[order[j]], steps = t->shape[order[j]] - 1;
    if (stride < span || stride > (INT64_MAX - span) / steps) return false;
    span += stride * steps;
  }
  return true;
}

bool rows_distinct(const va_tensor* t) { return places_distinct(t, t->ndim - 1, t->shape[t->ndim - 1]); }

namespace {

// The scales of a page-scaled cache that the call writes.
va_status check_written_scales(const va_tensor* t, int64_t num_blocks, int64_t hkv) {
  const va_status s = check_page_scales(t, num_blocks, hkv);
  return s == VA_OK && !places_distinct(t, 2, 1) ? VA_ERR_LAYOUT : s;
}

va_status check_rope(const va_rope* r, int64_t total_q, int64_t max_rot, AppendParams* p) {
  if (!r) return VA_OK;
  const va_tensor* t = r->cos_sin;
  if (!t) return VA_ERR_NULL;
  if (!dims_ok(t, 2)) return VA_ERR_SHAPE;
  if (t->dtype != VA_FP32) return VA_ERR_DTYPE;
  if (t->shape[0] < 1) return VA_ERR_SHAPE;
  if (t->shape[1] < 8 || t->shape[1] > max_rot || t->shape[1] % 8 != 0) return VA_ERR_UNSUPPORTED;
  if (r->interleaved != 0 && r->interleaved != 1) return VA_ERR_UNSUPPORTED;
  const va_status s = check_rows(t);
  if (s != VA_OK) return s;
  if (r->positions) {
    const va_tensor* q = r->positions;
    if (!dims_ok(q, 1) || q->shape[0] != total_q) return VA_ERR_SHAPE;
    if (q->dtype != VA_INT32) return VA_ERR_DTYPE;
    if (total_q > 1 && q->stride[0] != 1) return VA_ERR_LAYOUT;
    if (total_q > 0 && !q->data) return VA_ERR_NULL;
    p->positions = static_cast<const int32_t*>(q->data);
  }
  p->cos_sin = static_cast<const float*>(t->data);
  p->cs_s0 = t->stride[0];
  p->max_pos = t->shape[0];
  p->rot = (int32_t)t->shape[1];
  p->interleaved = r->interleaved;
  return VA_OK;
}

CacheView cache_view(const va_tensor* t, const va_tensor* scales) {
  CacheView c;
  c.data = t->data;
  c.s0 = t->stride[0];
  c.s1 = t->stride[1];
  c.s2 = t->stride[2];
  c.fp8 = t->dtype == VA_FP8_E4M3;
  c.scales = scales ? static_cast<float*>(scales->data) : nullptr;
  c.sc_s0 = scales ? scales->stride[0] : 0;
  c.sc_s1 = scales ? scales->stride[1] : 0;
  return c;
}

void set_batch(AppendParams* p, const va_tensor* bt, const va_tensor* cu, const va_tensor* su) {
  p->block_table = static_cast<const int32_t*>(bt->data);
  p->bt_s0 = bt->stride[0];
  p->bt_s1 = bt->stride[1];
  p->bt_width = (int32_t)bt->shape[1];
  p->cu_q = static_cast<const int32_t*>(cu->data);
  p->seqused_k = static_cast<const int32_t*>(su->data);
  p->num_seqs = (int32_t)su->shape[0];
}

// The weights of a norm over a head's columns.
va_status check_norm_weight(const va_tensor* t) {
  if (!t) return VA_OK;
  if (t->dtype != VA_BF16 && t->dtype != VA_FP32) return VA_ERR_DTYPE;
  if (!dims_ok(t, 1) || t->shape[0] != kHeadDim) return VA_ERR_SHAPE;
  if (t->stride[0] != 1) return VA_ERR_LAYOUT;
  if (!t->data) return VA_ERR_NULL;
  return aligned16(t->data) ? VA_OK : VA_ERR_LAYOUT;
}

va_status check_norm(const va_norm* n, AppendParams* p) {
  if (!n) return VA_OK;
  va_status s = check_norm_weight(n->q_weight);
  if (s == VA_OK) s = check_norm_weight(n->k_weight);
  if (s != VA_OK) return s;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps) || !std::isfinite(n->offset)) return VA_ERR_UNSUPPORTED;
  p->norm_eps = n->eps;
  p->norm_offset = n->offset;
  if (n->q_weight) {
    p->q_norm = n->q_weight->data;
    p->q_norm_fp32 = n->q_weight->dtype == VA_FP32;
  }
  if (n->k_weight) {
    p->k_norm = n->k_weight->data;
    p->k_norm_fp32 = n->k_weight->dtype == VA_FP32;
  }
  return VA_OK;
}

// q and q_out [total_q, hq, width]: both or neither, and only with something to do
// (a rotation, a norm).
va_status check_queries(const va_tensor* q, const va_tensor* q_out, int64_t total_q, int64_t width,
                        bool work, AppendParams* p) {
  if (!q && !q_out) return VA_OK;
  if (!q || !q_out || !work) return VA_ERR_NULL;
  if (!dims_ok(q, 3) || !dims_ok(q_out, 3)) return VA_ERR_SHAPE;
  if (q->dtype != VA_BF16 || q_out->dtype != VA_BF16) return VA_ERR_DTYPE;
  if (q->shape[2] != width) return VA_ERR_UNSUPPORTED;
  if (q->shape[0] != total_q || q->shape[1] < 1) return VA_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (q_out->shape[i] != q->shape[i]) return VA_ERR_SHAPE;
  va_status s = check_rows(q);
  if (s == VA_OK) s = check_rows(q_out);
  if (s != VA_OK) return s;
  if (!rows_distinct(q_out)) return VA_ERR_LAYOUT;
  if (q->shape[1] > INT32_MAX) return VA_ERR_UNSUPPORTED;
  p->q = static_cast<const uint16_t*>(q->data);
  p->q_s0 = q->stride[0];
  p->q_s1 = q->stride[1];
  p->q_out = static_cast<uint16_t*>(q_out->data);
  p->qo_s0 = q_out->stride[0];
  p->qo_s1 = q_out->stride[1];
  p->hq = (int32_t)q->shape[1];
  return VA_OK;
}

va_status run_append(const AppendParams& p, bool mla, void* stream) {
  const int64_t units = p.total_q / kPageSize + 2 * (int64_t)p.num_seqs;
  if (units > INT32_MAX || append_roles(mla, p) > 65535) return VA_ERR_UNSUPPORTED;
  if (p.total_q == 0 || p.num_seqs == 0) return VA_OK;  // no token
  return launch_append(p, mla, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}

}  // namespace

va_status check_page_scales(const va_tensor* t, int64_t num_blocks, int64_t hkv) {
  if (!dims_ok(t, 2) || t->shape[0] != num_blocks || t->shape[1] != hkv) return VA_ERR_SHAPE;
  if (t->dtype != VA_FP32) return VA_ERR_DTYPE;
  if ((num_blocks > 1 && t->stride[0] < 1) || (hkv > 1 && t->stride[1] < 1)) return VA_ERR_LAYOUT;
  if (numel(t) > 0 && !t->data) return VA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(t->data) & 3u) != 0) return VA_ERR_LAYOUT;
  return VA_OK;
}

}  // namespace va_host_impl

using namespace va_host_impl;

VA_EXPORT va_status verify_attn_append_kv(const va_tensor* q, const va_tensor* k, const va_tensor* v,
                                          const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                          const va_tensor* seqused_k, const va_rope* rope,
                                          const va_tensor* k_descale, const va_tensor* v_descale,
                                          va_tensor* k_scales, va_tensor* v_scales, va_tensor* q_out,
                                          va_tensor* k_cache, va_tensor* v_cache, void* stream) {
  return verify_attn_append_kv_norm(q, k, v, block_table, cu_seqlens_q, seqused_k, nullptr, rope, k_descale, v_descale,
                                    k_scales, v_scales, q_out, k_cache, v_cache, stream);
}

VA_EXPORT va_status verify_attn_append_kv_norm(const va_tensor* q, const va_tensor* k, const va_tensor* v,
                                               const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                               const va_tensor* seqused_k, const va_norm* norm, const va_rope* rope,
                                               const va_tensor* k_descale, const va_tensor* v_descale,
                                               va_tensor* k_scales, va_tensor* v_scales, va_tensor* q_out,
                                               va_tensor* k_cache, va_tensor* v_cache, void* stream) {
  if (!k || !v || !block_table || !cu_seqlens_q || !seqused_k || !k_cache || !v_cache) return VA_ERR_NULL;
  if (!dims_ok(k, 3) || !dims_ok(v, 3) || !dims_ok(k_cache, 4) || !dims_ok(v_cache, 4)) return VA_ERR_SHAPE;
  if (k->dtype != VA_BF16 || v->dtype != VA_BF16) return VA_ERR_DTYPE;
  if (k_cache->dtype != VA_FP8_E4M3 && k_cache->dtype != VA_BF16) return VA_ERR_DTYPE;
  if (v_cache->dtype != k_cache->dtype) return VA_ERR_DTYPE;
  if (k->shape[2] != va::kHeadDim || k_cache->shape[3] != va::kHeadDim || k_cache->shape[1] != va::kPageSize)
    return VA_ERR_UNSUPPORTED;
  for (int i = 0; i < 3; ++i)
    if (v->shape[i] != k->shape[i]) return VA_ERR_SHAPE;
  for (int i = 0; i < 4; ++i)
    if (v_cache->shape[i] != k_cache->shape[i]) return VA_ERR_SHAPE;
  const int64_t total_q = k->shape[0], hkv = k->shape[1];
  if (hkv < 1 || k_cache->shape[2] != hkv) return VA_ERR_SHAPE;
  if (total_q > INT32_MAX || hkv > INT32_MAX || k_cache->shape[0] > INT32_MAX) return VA_ERR_UNSUPPORTED;
  va_status s = check_batch(block_table, cu_seqlens_q, seqused_k);
  for (const va_tensor* t : {k, v, static_cast<const va_tensor*>(k_cache), static_cast<const va_tensor*>(v_cache)})
    if (s == VA_OK) s = check_rows(t);
  if (s != VA_OK) return s;
  if (!rows_distinct(k_cache) || !rows_distinct(v_cache)) return VA_ERR_LAYOUT;
  // K and V in one place (views that interleave have different addresses)
  if (k_cache->data && k_cache->data == v_cache->data) return VA_ERR_LAYOUT;
  if ((k_scales != nullptr) != (v_scales != nullptr)) return VA_ERR_NULL;
  if (k_scales) {
    if (k_cache->dtype != VA_FP8_E4M3) return VA_ERR_DTYPE;
    if (k_descale || v_descale) return VA_ERR_UNSUPPORTED;  // a page's scale is its descale
    s = check_written_scales(k_scales, k_cache->shape[0], hkv);
    if (s == VA_OK) s = check_written_scales(v_scales, k_cache->shape[0], hkv);
    if (s == VA_OK && k_scales->data && k_scales->data == v_scales->data) s = VA_ERR_LAYOUT;
  } else {
    s = check_descale(k_descale);
    if (s == VA_OK) s = check_descale(v_descale);
  }
  if (s != VA_OK) return s;
  va::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  s = check_rope(rope, total_q, va::kHeadDim, &p);
  if (s == VA_OK) s = check_norm(norm, &p);
  if (s == VA_OK) s = check_queries(q, q_out, total_q, va::kHeadDim, rope || p.q_norm, &p);
  if (s == VA_OK && p.q_norm && !q) s = VA_ERR_NULL;
  if (s != VA_OK) return s;
  p.k = static_cast<const uint16_t*>(k->data);
  p.k_s0 = k->stride[0];
  p.k_s1 = k->stride[1];
  p.v = static_cast<const uint16_t*>(v->data);
  p.v_s0 = v->stride[0];
  p.v_s1 = v->stride[1];
  p.kc = cache_view(k_cache, k_scales);
  p.vc = cache_view(v_cache, v_scales);
  p.k_descale = k_descale ? static_cast<const float*>(k_descale->data) : nullptr;
  p.v_descale = v_descale ? static_cast<const float*>(v_descale->data) : nullptr;
  set_batch(&p, block_table, cu_seqlens_q, seqused_k);
  p.total_q = (int32_t)total_q;
  p.hkv = (int32_t)hkv;
  p.num_blocks = (int32_t)k_cache->shape[0];
  return run_append(p, false, stream);
}

VA_EXPORT va_status verify_attn_append_mla(const va_tensor* q_pe, const va_tensor* latent, const va_tensor* k_pe,
                                           const va_tensor* block_table, const va_tensor* cu_seqlens_q,
                                           const va_tensor* seqused_k, const va_rope* rope,
                                           const va_tensor* descale, va_tensor* scales, va_tensor* q_pe_out,
                                           va_tensor* kv_cache, void* stream) {
  if (!latent || !k_pe || !block_table || !cu_seqlens_q || !seqused_k || !kv_cache) return VA_ERR_NULL;
  if (!dims_ok(latent, 2) || !dims_ok(k_pe, 2) || !dims_ok(kv_cache, 4)) return VA_ERR_SHAPE;
  if (latent->dtype != VA_BF16 || k_pe->dtype != VA_BF16) return VA_ERR_DTYPE;
  if (kv_cache->dtype != VA_FP8_E4M3 && kv_cache->dtype != VA_BF16) return VA_ERR_DTYPE;
  if (latent->shape[1] != va::kMlaNope || k_pe->shape[1] != va::kMlaPe || kv_cache->shape[1] != va::kPageSize ||
      kv_cache->shape[2] != 1 || kv_cache->shape[3] != va::kMlaRow)
    return VA_ERR_UNSUPPORTED;
  const int64_t total_q = latent->shape[0];
  if (k_pe->shape[0] != total_q) return VA_ERR_SHAPE;
  if (total_q > INT32_MAX || kv_cache->shape[0] > INT32_MAX) return VA_ERR_UNSUPPORTED;
  va_status s = check_batch(block_table, cu_seqlens_q, seqused_k);
  for (const va_tensor* t : {latent, k_pe, static_cast<const va_tensor*>(kv_cache)})
    if (s == VA_OK) s = check_rows(t);
  if (s != VA_OK) return s;
  if (!rows_distinct(kv_cache)) return VA_ERR_LAYOUT;
  if (scales) {
    if (kv_cache->dtype != VA_FP8_E4M3) return VA_ERR_DTYPE;
    if (descale) return VA_ERR_UNSUPPORTED;
    s = check_written_scales(scales, kv_cache->shape[0], 1);
  } else {
    s = check_descale(descale);
  }
  if (s != VA_OK) return s;
  va::AppendParams p;
  std::memset(&p, 0, sizeof(p));
  s = check_rope(rope, total_q, va::kMlaPe, &p);
  if (s == VA_OK && rope && p.rot != va::kMlaPe) s = VA_ERR_UNSUPPORTED;  // the whole rope part turns
  if (s == VA_OK) s = check_queries(q_pe, q_pe_out, total_q, va::kMlaPe, rope != nullptr, &p);
  if (s != VA_OK) return s;
  p.k = static_cast<const uint16_t*>(latent->data);
  p.k_s0 = latent->stride[0];
  p.v = static_cast<const uint16_t*>(k_pe->data);
  p.v_s0 = k_pe->stride[0];
  p.kc = cache_view(kv_cache, scales);
  p.k_descale = descale ? static_cast<const float*>(descale->data) : nullptr;
  set_batch(&p, block_table, cu_seqlens_q, seqused_k);
  p.total_q = (int32_t)total_q;
  p.hkv = 1;
  p.num_blocks = (int32_t)kv_cache->shape[0];
  return run_append(p, true, stream);
}
