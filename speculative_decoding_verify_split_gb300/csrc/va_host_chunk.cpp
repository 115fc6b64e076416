// Host side of the chunk attention (include/verify_attn.h): argument validation
// and the launch.
#include <climits>
#include <cmath>
#include <cstring>

#include "va_chunk.h"
#include "va_host_impl.h"

namespace va_host_impl {
namespace {

using namespace va;

// The units of the split and the row numbers stay inside their integers, also where prefix
// sums out of order give every sequence all rows of q.
bool fits(const Shapes& sh) {
  const int64_t group = sh.hq / sh.hkv;
  if (sh.total_q > (INT32_MAX - 2 * kChunkRows) / group) return false;
  const double rows = (double)sh.total_q * group;
  const double tiles = (rows / kChunkRows + 1.0) * (double)sh.num_seqs;
  const double cost = (double)sh.width * kPageSize * group + rows + 4.0 * kChunkKeys * group * kChunkItemCost;
  return sh.hkv * tiles * cost < 4611686018427387904.0;  // 2^62
}

va_status validate_chunk(const va_tensor* q, const va_tensor* k, const va_tensor* v, const va_tensor* ks, const va_tensor* vs,
                         const va_tensor* bt, const va_tensor* cu, const va_tensor* su, const va_tensor* kd,
                         const va_tensor* vd, const va_tensor* out, const va_options* opts, int32_t first_tokens,
                         Shapes* sh) {
  if (!q || !k || !v || !bt || !cu || !su || !out) return VA_ERR_NULL;
  if (!dims_ok(q, 3) || !dims_ok(k, 4) || !dims_ok(v, 4) || !dims_ok(out, 3)) return VA_ERR_SHAPE;
  if (q->dtype != VA_BF16 || out->dtype != VA_BF16) return VA_ERR_DTYPE;
  if ((k->dtype != VA_FP8_E4M3 && k->dtype != VA_BF16) || v->dtype != k->dtype) return VA_ERR_DTYPE;
  if (q->shape[2] != kHeadDim || k->shape[3] != kHeadDim || k->shape[1] != kPageSize) return VA_ERR_UNSUPPORTED;
  for (int i = 0; i < 4; ++i)
    if (v->shape[i] != k->shape[i]) return VA_ERR_SHAPE;
  for (int i = 0; i < 3; ++i)
    if (out->shape[i] != q->shape[i]) return VA_ERR_SHAPE;
  const int64_t hq = q->shape[1], hkv = k->shape[2];
  if (hq < 1 || hkv < 1 || hq % hkv != 0) return VA_ERR_SHAPE;
  va_status s = check_batch(bt, cu, su);
  for (const va_tensor* t : {q, k, v, out})
    if (s == VA_OK) s = check_rows(t);
  if (s != VA_OK) return s;
  if (!rows_distinct(out)) return VA_ERR_LAYOUT;
  for (const va_tensor* t : {bt, cu, su, opts ? opts->sinks : nullptr})
    if (t && (reinterpret_cast<uintptr_t>(t->data) & 3u) != 0) return VA_ERR_LAYOUT;
  if ((ks != nullptr) != (vs != nullptr)) return VA_ERR_NULL;
  if (ks) {
    if (k->dtype != VA_FP8_E4M3) return VA_ERR_DTYPE;
    if (kd || vd) return VA_ERR_UNSUPPORTED;  // a page's scale is its descale
    s = check_page_scales(ks, k->shape[0], hkv);
    if (s == VA_OK) s = check_page_scales(vs, k->shape[0], hkv);
  } else {
    s = check_descale(kd);
    if (s == VA_OK) s = check_descale(vd);
  }
  if (s != VA_OK) return s;
  sh->total_q = q->shape[0];
  sh->hq = hq;
  sh->hkv = hkv;
  sh->num_blocks = k->shape[0];
  sh->num_seqs = su->shape[0];
  sh->width = bt->shape[1];
  sh->kv_dtype = k->dtype;
  s = validate_options(opts, *sh);
  if (s != VA_OK) return s;
  if (first_tokens < 0) return VA_ERR_UNSUPPORTED;
  if (hq > INT32_MAX || hkv > INT32_MAX || sh->num_blocks >= INT32_MAX || !fits(*sh)) return VA_ERR_UNSUPPORTED;
  return VA_OK;
}

}  // namespace
}  // namespace va_host_impl

using namespace va_host_impl;

VA_EXPORT size_t verify_attn_chunk_workspace_size(void) {
  LibraryCall call;
  if (begin_call(&call) != VA_OK || call.chunk_pairs < 1) return 0;
  return va::chunk_workspace(call.chunk_pairs).total;
}

VA_EXPORT va_status verify_attn_chunk(const va_tensor* q, const va_tensor* k_cache, const va_tensor* v_cache,
                                      const va_tensor* k_scales, const va_tensor* v_scales, const va_tensor* block_table,
                                      const va_tensor* cu_seqlens_q, const va_tensor* seqused_k, float softmax_scale,
                                      const va_tensor* k_descale, const va_tensor* v_descale, va_tensor* out,
                                      const va_options* opts, int32_t first_tokens, void* workspace,
                                      size_t workspace_bytes, int32_t num_splits, void* stream) {
  Shapes sh;
  va_status s = validate_chunk(q, k_cache, v_cache, k_scales, v_scales, block_table, cu_seqlens_q, seqused_k, k_descale,
                               v_descale, out, opts, first_tokens, &sh);
  if (s != VA_OK) return s;
  if (num_splits < 0) return VA_ERR_UNSUPPORTED;
  const bool library_status = (num_splits & VA_LIBRARY_STATUS) != 0;
  if (sh.total_q == 0 || sh.num_seqs == 0) return VA_OK;
  LibraryCall call;
  s = begin_call(&call);
  if (s != VA_OK) return s;
  if (call.chunk_pairs < 1) return VA_ERR_UNSUPPORTED;
  const va::ChunkWorkspace lay = va::chunk_workspace(call.chunk_pairs);
  s = take_workspace(&call, &workspace, &workspace_bytes, lay.total, static_cast<cudaStream_t>(stream));
  if (s != VA_OK) return s;
  if (workspace_bytes < lay.total || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return VA_ERR_WORKSPACE;
  va::ChunkParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(q->data);
  p.q_s0 = q->stride[0];
  p.q_s1 = q->stride[1];
  p.block_table = static_cast<const int32_t*>(block_table->data);
  p.bt_s0 = block_table->stride[0];
  p.bt_s1 = block_table->stride[1];
  p.bt_width = (int32_t)sh.width;
  p.cu_q = static_cast<const int32_t*>(cu_seqlens_q->data);
  p.seqused_k = static_cast<const int32_t*>(seqused_k->data);
  p.k_descale = k_descale ? static_cast<const float*>(k_descale->data) : nullptr;
  p.v_descale = v_descale ? static_cast<const float*>(v_descale->data) : nullptr;
  if (k_scales) {
    p.k_scales = static_cast<const float*>(k_scales->data);
    p.ks_s0 = k_scales->stride[0];
    p.ks_s1 = k_scales->stride[1];
    p.v_scales = static_cast<const float*>(v_scales->data);
    p.vs_s0 = v_scales->stride[0];
    p.vs_s1 = v_scales->stride[1];
  }
  p.sinks = opts && opts->sinks ? static_cast<const float*>(opts->sinks->data) : nullptr;
  p.out = static_cast<uint16_t*>(out->data);
  p.o_s0 = out->stride[0];
  p.o_s1 = out->stride[1];
  p.out_v8 = (reinterpret_cast<uintptr_t>(out->data) & 31u) == 0 && (p.o_s0 * 2) % 32 == 0 && (p.o_s1 * 2) % 32 == 0;
  p.num_seqs = (int32_t)sh.num_seqs;
  p.hq = (int32_t)sh.hq;
  p.hkv = (int32_t)sh.hkv;
  p.group = (int32_t)(sh.hq / sh.hkv);
  if (p.group > 1) {
    int log2 = 1;
    while ((1ll << log2) < p.group) ++log2;
    p.group_m = (uint32_t)((1ull << (31 + log2)) / (uint32_t)p.group + 1);
    p.group_s = (uint32_t)(log2 - 1);
  }
  p.num_blocks = (int32_t)sh.num_blocks;
  p.total_q = (int32_t)sh.total_q;
  p.kv_fp8 = sh.kv_dtype == VA_FP8_E4M3;
  p.scale_log2 = (float)((double)softmax_scale * 1.4426950408889634);
  p.softcap_log2 = opts ? (float)((double)opts->softcap * 1.4426950408889634) : 0.f;
  p.window_left = opts ? opts->window_left : -1;
  p.first_tokens = p.window_left >= 0 ? first_tokens : 0;
  p.pairs = call.chunk_pairs;
  p.force = num_splits & ~VA_LIBRARY_STATUS;
  p.wait_limit_ns = wait_limit_ns();
  char* base = static_cast<char*>(workspace);
  p.ws_status = library_status ? call.status : reinterpret_cast<int32_t*>(base);
  p.ws_start = reinterpret_cast<va::ChunkStart*>(base + lay.start_off);
  p.ws_ml = reinterpret_cast<float*>(base + lay.ml_off);
  p.ws_acc = reinterpret_cast<float*>(base + lay.acc_off);
  CUtensorMap tm_k, tm_v;
  std::memset(&tm_k, 0, sizeof(tm_k));
  std::memset(&tm_v, 0, sizeof(tm_v));
  if (sh.num_blocks > 0 &&  // an empty cache has no page to load
      (!make_kv_map(&tm_k, k_cache, sh.num_blocks, sh.hkv) || !make_kv_map(&tm_v, v_cache, sh.num_blocks, sh.hkv)))
    return VA_ERR_LAYOUT;
  return va::launch_chunk(p, tm_k, tm_v, static_cast<cudaStream_t>(stream)) == cudaSuccess ? VA_OK : VA_ERR_CUDA;
}
