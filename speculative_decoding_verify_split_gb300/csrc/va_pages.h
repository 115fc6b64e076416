// Launch parameters of the page pool's kernels (va_pages.cu). Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "va_internal.h"

namespace va {

// Status bits (VA_PG_*).
constexpr int32_t kPgBadSeq = 1, kPgInUse = 2, kPgNoPages = 4, kPgRowFull = 8, kPgBadTable = 16;

constexpr int kPoolCtas = 8;             // one cluster
constexpr int kPoolThreads = 1024;
constexpr int64_t kMaxPoolPages = 1 << 22;
constexpr int64_t kMaxPoolSeqs = 8192;

// Sequences whose pages are counted: block table [num_seqs, width], lengths, pages a row
// holds, sequences that hold a page.
struct PoolParams {
  int32_t* table;
  int64_t t_s0, t_s1;
  int32_t* seqused;
  int32_t* page_count;
  int32_t* refs;
  int32_t num_seqs, width, num_pages;
  int32_t* status;          // nullable
  const int32_t* list;      // free: sequences; fork: parents
  const int32_t* children;  // fork
  int32_t n;                // entries of the list
  const int32_t* new_tokens;  // reserve
  int32_t* src;
  int32_t* dst;
  int32_t* room;
};

// A CTA of the copy moves kCopyThreads * kCopyUnits 16-byte units of a page; a launch has at
// most 65,535 of them a page, which is what a token row may hold.
constexpr int kCopyThreads = 128, kCopyUnits = 4;
constexpr int64_t kMaxCopyRowUnits = 65535ll * kCopyThreads * kCopyUnits / kPageSize;

// One cache whose pages are copied: a page is 16 x heads rows of `units` 16-byte units.
struct PageView {
  char* data;               // null: none
  int64_t s0, s1, s2;       // bytes
  float* scales;            // nullable
  int64_t sc_s0, sc_s1;
};

struct CopyParams {
  PageView c[2];
  const int32_t* src;
  const int32_t* dst;
  int32_t n, heads, units, num_pages;
};

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream);
cudaError_t launch_free_pages(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_fork_pages(const PoolParams& p, cudaStream_t stream);
cudaError_t launch_reserve_pages(const PoolParams& p, cudaStream_t stream);

}  // namespace va
