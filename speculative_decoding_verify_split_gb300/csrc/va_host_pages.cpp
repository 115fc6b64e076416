// Host side of the page pool's entry points (include/verify_attn.h): argument
// validation and the launches.
#include <climits>
#include <cstring>
#include <initializer_list>

#include "va_host_impl.h"
#include "va_pages.h"

namespace va_host_impl {
namespace {

using namespace va;

static_assert(kPgBadSeq == VA_PG_BAD_SEQ && kPgInUse == VA_PG_IN_USE && kPgNoPages == VA_PG_NO_PAGES &&
                  kPgRowFull == VA_PG_ROW_FULL && kPgBadTable == VA_PG_BAD_TABLE,
              "status bits");

// A contiguous int32 vector.
va_status check_ints(const va_tensor* t, int64_t n) {
  if (!dims_ok(t, 1) || (n >= 0 && t->shape[0] != n)) return VA_ERR_SHAPE;
  if (t->dtype != VA_INT32) return VA_ERR_DTYPE;
  if (t->shape[0] > INT32_MAX) return VA_ERR_UNSUPPORTED;
  if (t->shape[0] > 1 && t->stride[0] != 1) return VA_ERR_LAYOUT;
  if (t->shape[0] > 0 && !t->data) return VA_ERR_NULL;
  return (reinterpret_cast<uintptr_t>(t->data) & 3u) != 0 ? VA_ERR_LAYOUT : VA_OK;
}

// Whether a written vector has its place to itself: none of `n` others reaches into it.
bool apart(const va_tensor* t, const va_tensor* const* others, int n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(t->data), e = a + 4 * (uintptr_t)t->shape[0];
  for (int i = 0; i < n; ++i) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(others[i]->data), f = b + 4 * (uintptr_t)others[i]->shape[0];
    if (a < f && b < e && a < e && b < f) return false;
  }
  return true;
}

// The last `fresh` of the vectors, and the first three, are written; those between are read.
bool all_apart(std::initializer_list<const va_tensor*> v, int fresh) {
  const int n = (int)v.size();
  for (int i = 0; i < n; ++i) {
    const bool written = i < 3 || i >= n - fresh;
    const va_tensor* const* t = v.begin();
    if (written && !(apart(t[i], t, i) && apart(t[i], t + i + 1, n - i - 1))) return false;
  }
  return true;
}

va_status check_pool(const va_tensor* bt, const va_tensor* su, const va_tensor* pc, const va_tensor* refs, int32_t* status,
                     PoolParams* p) {
  std::memset(p, 0, sizeof(*p));
  if (!bt || !su || !pc || !refs) return VA_ERR_NULL;
  if (!dims_ok(bt, 2)) return VA_ERR_SHAPE;
  if (bt->dtype != VA_INT32) return VA_ERR_DTYPE;
  if (bt->shape[0] > INT32_MAX || bt->shape[1] > INT32_MAX / kPageSize) return VA_ERR_UNSUPPORTED;
  if (numel(bt) > 0 && !bt->data) return VA_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(bt->data) & 3u) != 0) return VA_ERR_LAYOUT;
  va_status s = check_ints(su, bt->shape[0]);
  if (s == VA_OK) s = check_ints(pc, bt->shape[0]);
  if (s == VA_OK) s = check_ints(refs, -1);
  if (s != VA_OK) return s;
  if (!places_distinct(bt, 2, 1)) return VA_ERR_LAYOUT;
  if ((reinterpret_cast<uintptr_t>(status) & 3u) != 0) return VA_ERR_LAYOUT;
  p->table = static_cast<int32_t*>(bt->data);
  p->t_s0 = bt->stride[0];
  p->t_s1 = bt->stride[1];
  p->seqused = static_cast<int32_t*>(su->data);
  p->page_count = static_cast<int32_t*>(pc->data);
  p->refs = static_cast<int32_t*>(refs->data);
  p->num_seqs = (int32_t)bt->shape[0];
  p->width = (int32_t)bt->shape[1];
  p->num_pages = (int32_t)refs->shape[0];
  p->status = status;
  return VA_OK;
}

// One cache of copy_pages.
va_status check_copied(const va_tensor* t, const va_tensor* scales, PageView* v) {
  if (!dims_ok(t, 4)) return VA_ERR_SHAPE;
  if (t->dtype != VA_BF16 && t->dtype != VA_FP8_E4M3) return VA_ERR_DTYPE;
  const int64_t es = t->dtype == VA_BF16 ? 2 : 1;
  if (t->shape[1] != kPageSize || t->shape[3] * es % 16 != 0 || t->shape[0] > INT32_MAX || t->shape[2] < 1 || t->shape[3] < 1 ||
      t->shape[2] > kMaxCopyRowUnits / (t->shape[3] * es / 16))
    return VA_ERR_UNSUPPORTED;
  va_status s = check_rows(t);
  if (s != VA_OK) return s;
  if (!rows_distinct(t)) return VA_ERR_LAYOUT;
  v->data = static_cast<char*>(t->data);
  v->s0 = t->stride[0] * es;
  v->s1 = t->stride[1] * es;
  v->s2 = t->stride[2] * es;
  if (scales) {
    if (t->dtype != VA_FP8_E4M3) return VA_ERR_DTYPE;
    s = check_page_scales(scales, t->shape[0], t->shape[2]);
    if (s != VA_OK) return s;
    if (!places_distinct(scales, 2, 1)) return VA_ERR_LAYOUT;
    v->scales = static_cast<float*>(scales->data);
    v->sc_s0 = scales->stride[0];
    v->sc_s1 = scales->stride[1];
  }
  return VA_OK;
}

va_status launched(cudaError_t e) { return e == cudaSuccess ? VA_OK : VA_ERR_CUDA; }

}  // namespace
}  // namespace va_host_impl

using namespace va_host_impl;

VA_EXPORT va_status verify_attn_copy_pages(va_tensor* k_cache, va_tensor* v_cache, va_tensor* k_scales, va_tensor* v_scales,
                                           const va_tensor* src, const va_tensor* dst, void* stream) {
  if (!k_cache || !src || !dst) return VA_ERR_NULL;
  if (v_cache ? (k_scales != nullptr) != (v_scales != nullptr) : v_scales != nullptr) return VA_ERR_NULL;
  va::CopyParams p;
  std::memset(&p, 0, sizeof(p));
  va_status s = check_copied(k_cache, k_scales, &p.c[0]);
  if (s != VA_OK) return s;
  if (v_cache) {
    s = check_copied(v_cache, v_scales, &p.c[1]);
    if (s != VA_OK) return s;
    if (v_cache->dtype != k_cache->dtype) return VA_ERR_DTYPE;
    for (int i = 0; i < 4; ++i)
      if (v_cache->shape[i] != k_cache->shape[i]) return VA_ERR_SHAPE;
    if (k_cache->data && k_cache->data == v_cache->data) return VA_ERR_LAYOUT;
    if (k_scales && k_scales->data && k_scales->data == v_scales->data) return VA_ERR_LAYOUT;
  }
  s = check_ints(src, -1);
  if (s == VA_OK) s = check_ints(dst, src->shape[0]);
  if (s != VA_OK) return s;
  p.src = static_cast<const int32_t*>(src->data);
  p.dst = static_cast<const int32_t*>(dst->data);
  p.n = (int32_t)src->shape[0];
  p.heads = (int32_t)k_cache->shape[2];
  p.units = (int32_t)(k_cache->shape[3] * (k_cache->dtype == VA_BF16 ? 2 : 1) / 16);
  p.num_pages = (int32_t)k_cache->shape[0];
  if (p.n == 0 || p.num_pages == 0) return VA_OK;
  return launched(va::launch_copy_pages(p, static_cast<cudaStream_t>(stream)));
}

VA_EXPORT va_status verify_attn_free_pages(const va_tensor* block_table, va_tensor* seqused_k, va_tensor* page_count,
                                           va_tensor* refs, const va_tensor* seqs, int32_t* status, void* stream) {
  va::PoolParams p;
  va_status s = check_pool(block_table, seqused_k, page_count, refs, status, &p);
  if (s != VA_OK) return s;
  if (!seqs) return VA_ERR_NULL;
  s = check_ints(seqs, -1);
  if (s != VA_OK) return s;
  if (!all_apart({seqused_k, page_count, refs, seqs}, 0)) return VA_ERR_LAYOUT;
  p.list = static_cast<const int32_t*>(seqs->data);
  p.n = (int32_t)seqs->shape[0];
  if (p.n == 0) return VA_OK;
  return launched(va::launch_free_pages(p, static_cast<cudaStream_t>(stream)));
}

VA_EXPORT va_status verify_attn_fork_pages(va_tensor* block_table, va_tensor* seqused_k, va_tensor* page_count,
                                           va_tensor* refs, const va_tensor* parents, const va_tensor* children,
                                           int32_t* status, void* stream) {
  va::PoolParams p;
  va_status s = check_pool(block_table, seqused_k, page_count, refs, status, &p);
  if (s != VA_OK) return s;
  if (!parents || !children) return VA_ERR_NULL;
  s = check_ints(parents, -1);
  if (s == VA_OK) s = check_ints(children, parents->shape[0]);
  if (s != VA_OK) return s;
  if (!all_apart({seqused_k, page_count, refs, parents, children}, 0)) return VA_ERR_LAYOUT;
  p.list = static_cast<const int32_t*>(parents->data);
  p.children = static_cast<const int32_t*>(children->data);
  p.n = (int32_t)parents->shape[0];
  if (p.n == 0) return VA_OK;
  return launched(va::launch_fork_pages(p, static_cast<cudaStream_t>(stream)));
}

VA_EXPORT va_status verify_attn_reserve_pages(va_tensor* block_table, const va_tensor* seqused_k, va_tensor* page_count,
                                              va_tensor* refs, const va_tensor* new_tokens, va_tensor* src, va_tensor* dst,
                                              va_tensor* room, int32_t* status, void* stream) {
  va::PoolParams p;
  va_status s = check_pool(block_table, seqused_k, page_count, refs, status, &p);
  if (s != VA_OK) return s;
  if (!new_tokens || !src || !dst || !room) return VA_ERR_NULL;
  for (const va_tensor* t : {new_tokens, static_cast<const va_tensor*>(src), static_cast<const va_tensor*>(dst),
                             static_cast<const va_tensor*>(room)}) {
    s = check_ints(t, p.num_seqs);
    if (s != VA_OK) return s;
  }
  if (p.num_seqs > va::kMaxPoolSeqs || p.num_pages > va::kMaxPoolPages) return VA_ERR_UNSUPPORTED;
  if (!all_apart({seqused_k, page_count, refs, new_tokens, src, dst, room}, 3)) return VA_ERR_LAYOUT;
  p.new_tokens = static_cast<const int32_t*>(new_tokens->data);
  p.src = static_cast<int32_t*>(src->data);
  p.dst = static_cast<int32_t*>(dst->data);
  p.room = static_cast<int32_t*>(room->data);
  if (p.num_seqs == 0) return VA_OK;
  return launched(va::launch_reserve_pages(p, static_cast<cudaStream_t>(stream)));
}
