// Launch parameters of the chunk attention (va_chunk.cu), and the split of its
// work, shared by the main and the merge kernel. Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "va_internal.h"

namespace va {

constexpr int kChunkRows = 256;  // packed rows of a work item: 128 per CTA of the pair
constexpr int kChunkKeys = 128;  // keys of a tile
// Cost of an item beside its tiles, in tiles: Q's load, the pipeline's refill and the
// epilogue; at least 3 (see chunk_cost). A prompt of 8,192 tokens (16 query and 2 KV heads)
// and four of 700 to 2,500: 3 tiles 379 and 126 us, 4 362 and 123, 5 333 and 117, 6 341 and
// 119, 7 335 and 120.
constexpr int kChunkItemCost = 5;

struct ChunkParams {
  const uint16_t* q;  // [total_q, hq, 256] bf16 bits
  int64_t q_s0, q_s1;
  const int32_t* block_table;
  int64_t bt_s0, bt_s1;
  int32_t bt_width;
  const int32_t* cu_q;
  const int32_t* seqused_k;
  const float* k_descale;  // nullable
  const float* v_descale;  // nullable
  const float* k_scales;   // [num_blocks, hkv], a page-scaled cache; else null
  const float* v_scales;
  int64_t ks_s0, ks_s1, vs_s0, vs_s1;
  const float* sinks;      // nullable, [hq]
  uint16_t* out;           // [total_q, hq, 256] bf16 bits
  int64_t o_s0, o_s1;
  int32_t out_v8;          // 32-byte stores fit out
  int32_t num_seqs, hq, hkv, group, num_blocks, total_q;
  uint32_t group_m, group_s;  // division by group (by_group)
  int32_t kv_fp8;
  float scale_log2;        // softmax_scale * log2(e)
  float softcap_log2;      // 0: none
  int32_t window_left;     // -1: none
  int32_t first_tokens;    // with a window: keys [0, first_tokens) stay visible
  int32_t pairs;           // CTA pairs of the launch
  int32_t force;           // > 0: split over this many of them
  uint64_t wait_limit_ns;
  int32_t* ws_status;
  struct ChunkStart* ws_start;  // [pairs]
  float* ws_ml;            // [2 * pairs][256][2]: reference (log2 units), row sum
  float* ws_acc;           // [2 * pairs][256][256]: unnormalised output rows
};

// Where a pair's share of the work starts: row tile m of head h of sequence b,
// whose first unit is `off`. total: all units; used: pairs that share them (0 in the first
// pair's: nothing to join; a pair that has an item to itself counts from the item on).
struct ChunkStart {
  int64_t off, total;
  int32_t b, h, m, used;
};

struct ChunkWorkspace {
  size_t start_off, ml_off, acc_off, total;
};

inline ChunkWorkspace chunk_workspace(int64_t pairs) {
  ChunkWorkspace w;
  w.start_off = 256;  // the status word ahead
  w.ml_off = w.start_off + align_up(sizeof(ChunkStart) * (size_t)pairs, 256);
  w.acc_off = w.ml_off + align_up(sizeof(float) * 2 * 2 * (size_t)pairs * kChunkRows, 256);
  w.total = w.acc_off + sizeof(float) * 2 * (size_t)pairs * kChunkRows * kHeadDim;
  return w;
}

cudaError_t prepare_chunk(int32_t* max_pairs);
cudaError_t launch_chunk(const ChunkParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream);

}  // namespace va
