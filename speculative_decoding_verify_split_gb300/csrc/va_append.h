// Launch parameters of the append kernels (va_append.cu). Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "va_internal.h"

namespace va {

// A paged cache [num_blocks, 16, heads, width] that is written; strides in
// elements. scales: per page and KV head (fp32), or null.
struct CacheView {
  void* data;
  int64_t s0, s1, s2;
  int32_t fp8;
  float* scales;
  int64_t sc_s0, sc_s1;
};

struct AppendParams {
  const uint16_t* q;  // [total_q, hq, 256 or 64] bf16 bits; null with hq == 0
  int64_t q_s0, q_s1;
  uint16_t* q_out;
  int64_t qo_s0, qo_s1;
  const uint16_t* k;  // [total_q, hkv, 256], or the latent [total_q, 512]
  int64_t k_s0, k_s1;
  const uint16_t* v;  // [total_q, hkv, 256], or the rope key [total_q, 64]
  int64_t v_s0, v_s1;
  CacheView kc, vc;   // a latent cache is kc alone
  const int32_t* block_table;
  int64_t bt_s0, bt_s1;
  int32_t bt_width;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const int32_t* positions;  // nullable: S - L + t
  const float* cos_sin;      // [max_pos, rot]: cos | sin; null: no rotation (rot == 0)
  int64_t cs_s0;
  int64_t max_pos;
  int32_t rot;
  int32_t interleaved;
  // Norms of queries and keys (verify_attn_append_kv_norm): the weights of a head's 256
  // columns, bf16 bits or fp32, plus norm_offset; null: not normalised
  const void* q_norm;
  const void* k_norm;
  int32_t q_norm_fp32, k_norm_fp32;
  float norm_eps, norm_offset;
  const float* k_descale;    // nullable
  const float* v_descale;    // nullable
  int32_t num_seqs, total_q, hq, hkv, num_blocks;
};

// CTAs per page (grid.y).
int64_t append_roles(bool mla, const AppendParams& p);
cudaError_t launch_append(const AppendParams& p, bool mla, cudaStream_t stream);

}  // namespace va
