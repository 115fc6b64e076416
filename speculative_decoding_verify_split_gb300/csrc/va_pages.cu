// Pages of the caches: copies, and the pool that sequences share them from.
//
// The pool is three arrays beside the block table: seqused (tokens), page_count (pages
// that a row holds) and refs (rows that hold a page; 0: free). A fork gives a new row
// its parent's pages and counts them once more. Before a sequence writes on, `reserve`
// gives it pages of its own for what it will write: a page in that range that other
// rows hold too is replaced (the caller copies its contents, one page a sequence at
// most: only the page of the next token holds tokens), and rows grow. Everything is
// decided from the arrays as they are at the call's start, in the order of sequences and
// of places in their rows, and the k-th page needed is the k-th free one, so results do
// not depend on timing.
#include "va_pages.h"
#include "va_ptx.cuh"

namespace va {
namespace {

__device__ __forceinline__ void report(const PoolParams& p, int32_t bit) {
  if (p.status) atomicOr(p.status, bit);
}

// ---- copies ------------------------------------------------------------------------------
//
// A CTA moves 8 KB of one cache's page, four 16-byte units a thread, all loads ahead of
// the stores. The bound is memory, both directions: 258 MB in 40.6 us, 94 % of the
// measured copy bandwidth; a few pages are latency, 3.0 us.
__global__ void __launch_bounds__(kCopyThreads, 16) va_copy_pages_kernel(const CopyParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x;
  const int src = p.src[i], dst = p.dst[i];
  if ((unsigned)src >= (unsigned)p.num_pages || (unsigned)dst >= (unsigned)p.num_pages || src == dst) return;
  const PageView& c = p.c[blockIdx.z];
  const char* from = c.data + (int64_t)src * c.s0;
  char* to = c.data + (int64_t)dst * c.s0;
  const int rows = kPageSize * p.heads, total = rows * p.units;
  const int u0 = blockIdx.y * (kCopyThreads * kCopyUnits) + threadIdx.x;
  const bool flat = c.s2 == (int64_t)p.units * 16 && c.s1 == c.s2 * p.heads;
  uint4 v[kCopyUnits];
  int64_t at[kCopyUnits];
#pragma unroll
  for (int k = 0; k < kCopyUnits; ++k) {
    const int u = u0 + k * kCopyThreads;
    if (flat) {
      at[k] = (int64_t)u * 16;
    } else {
      const int row = u / p.units, t = row / p.heads;
      at[k] = t * c.s1 + (int64_t)(row - t * p.heads) * c.s2 + (int64_t)(u - row * p.units) * 16;
    }
    if (u < total) v[k] = *reinterpret_cast<const uint4*>(from + at[k]);
  }
#pragma unroll
  for (int k = 0; k < kCopyUnits; ++k)
    if (u0 + k * kCopyThreads < total) *reinterpret_cast<uint4*>(to + at[k]) = v[k];
  if (c.scales && blockIdx.y == 0)
    for (int h = threadIdx.x; h < p.heads; h += kCopyThreads)
      c.scales[(int64_t)dst * c.sc_s0 + (int64_t)h * c.sc_s1] = c.scales[(int64_t)src * c.sc_s0 + (int64_t)h * c.sc_s1];
}

// ---- free --------------------------------------------------------------------------------
//
// A CTA a listed sequence. Whoever takes the row's count first frees it: a sequence listed
// twice is freed once.
constexpr int kRowThreads = 256;

__global__ void __launch_bounds__(kRowThreads) va_free_pages_kernel(const PoolParams p) {
  __shared__ int s_count;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = p.list[blockIdx.x];
  if ((unsigned)b >= (unsigned)p.num_seqs) {
    if (threadIdx.x == 0) report(p, kPgBadSeq);
    return;
  }
  const int* row = p.table + (int64_t)b * p.t_s0;
  // the first entries are under way beside the count
  const int early = (int)threadIdx.x < p.width ? row[(int64_t)threadIdx.x * p.t_s1] : 0;
  if (threadIdx.x == 0) {
    // (a count that no row has stays: nobody writes it, so every listing sees it)
    int n = *static_cast<const volatile int*>(p.page_count + b);
    if (n < 0 || n > p.width) {
      report(p, kPgBadTable);
      n = 0;
    } else {
      n = atomicExch(p.page_count + b, 0);
      p.seqused[b] = 0;
    }
    s_count = n;
  }
  __syncthreads();
#pragma unroll 4
  for (int j = threadIdx.x; j < s_count; j += kRowThreads) {
    const int page = j < kRowThreads ? early : row[(int64_t)j * p.t_s1];
    if ((unsigned)page >= (unsigned)p.num_pages) {
      report(p, kPgBadTable);
      continue;
    }
    if (atomicSub(p.refs + page, 1) <= 0) {  // nobody held it
      atomicAdd(p.refs + page, 1);
      report(p, kPgBadTable);
    }
  }
}

// ---- fork --------------------------------------------------------------------------------
//
// A CTA a child. A child listed a second time, or listed as a parent too, is refused: its
// row would be written and read in one call.
__global__ void __launch_bounds__(kRowThreads) va_fork_pages_kernel(const PoolParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i = blockIdx.x;
  const int parent = p.list[i], child = p.children[i];
  bool bad = (unsigned)parent >= (unsigned)p.num_seqs || (unsigned)child >= (unsigned)p.num_seqs;
  for (int j = threadIdx.x; j < p.n; j += kRowThreads)
    bad |= p.list[j] == child || (j < i && p.children[j] == child);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(p, kPgBadSeq);
    return;
  }
  // (read by every thread before thread 0 writes the child's)
  const int used = p.seqused[parent], held = p.page_count[parent], in_use = p.page_count[child];
  const int64_t n64 = ((int64_t)used + kPageSize - 1) / kPageSize;
  __syncthreads();
  if (used < 0 || n64 > held || n64 > p.width || in_use != 0) {
    if (threadIdx.x == 0) report(p, in_use != 0 ? kPgInUse : kPgBadTable);
    return;
  }
  const int n = (int)n64;
  if (threadIdx.x == 0) {
    p.page_count[child] = n;
    p.seqused[child] = used;
  }
  const int* from = p.table + (int64_t)parent * p.t_s0;
  int* to = p.table + (int64_t)child * p.t_s0;
#pragma unroll 4
  for (int j = threadIdx.x; j < n; j += kRowThreads) {
    const int page = from[(int64_t)j * p.t_s1];
    to[(int64_t)j * p.t_s1] = page;
    if ((unsigned)page < (unsigned)p.num_pages)
      atomicAdd(p.refs + page, 1);
    else
      report(p, kPgBadTable);
  }
}

// ---- reserve -----------------------------------------------------------------------------
//
// One cluster of eight CTAs, a thousand threads each, so that the pool is read in a few
// loads a thread and the parts meet on chip: a bitmap of the free pages in shared memory,
// an eighth of the pool a CTA, with the number of free pages ahead of each word. Steps,
// between cluster barriers:
//  1  every CTA: each sequence's needs and their prefix sums; its part of the bitmap;
//  2  a sequence's thread marks the shared places of its row (as ~page);
//  3  a free page's thread puts it in its place, where it grows a row, or hands it to the
//     sequence; then a sequence's thread replaces its marked places (the first by that
//     page, others by the pages of their ranks) and gives up the shared ones;
//  4  counts of the rows.
// It is latency: three dependent loads, the scans and four barriers.
struct Want {
  int first, have, want;  // places to write: [first, want), the row holding `have`
  bool ok;                // something to reserve, in a row that is wide enough
};

__device__ __forceinline__ Want wants(const PoolParams& p, int b, bool tell) {
  Want w;
  const int used = p.seqused[b], add = p.new_tokens[b];
  w.have = p.page_count[b];
  w.ok = add > 0;
  const bool bad = used < 0 || w.have < 0 || w.have > p.width;
  const int64_t want = ((int64_t)used + add + kPageSize - 1) / kPageSize;
  if (w.ok && (bad || want > p.width)) {
    if (tell) report(p, bad ? kPgBadTable : kPgRowFull);
    w.ok = false;
  }
  w.first = used < 0 ? 0 : used / kPageSize;
  w.want = w.ok ? (int)want : 0;
  if (w.ok && w.first + (used % kPageSize != 0) > w.have) {  // tokens without pages
    if (tell) report(p, kPgBadTable);
    w.ok = false;
    w.want = 0;
  }
  return w;
}

__device__ __forceinline__ bool is_shared(const PoolParams& p, int page) {
  return (unsigned)page < (unsigned)p.num_pages && p.refs[page] > 1;
}

// Inclusive sums of one value a thread over the CTA; *total: the CTA's.
__device__ __forceinline__ int64_t block_inclusive(int64_t v, int64_t* scratch, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  if (warp > 0) v += scratch[warp - 1];
  *total = scratch[31];
  __syncthreads();
  return v;
}

__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  ptx::cluster_arrive();
  __syncwarp();
  ptx::cluster_wait();
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Dynamic shared memory: the words of this CTA's part of the bitmap, the free pages ahead
// of each of them (in the part), the sequences' sums [num_seqs + 1], a bit for each that is
// refused and one for each that needs pages (sums that saturate are equal, too).
__global__ void __launch_bounds__(kPoolThreads, 1) va_reserve_pages_kernel(const PoolParams p, int words) {
  extern __shared__ int32_t dyn[];
  __shared__ int64_t scratch[32];
  __shared__ int s_free;  // free pages of this CTA's part
  uint32_t* map = reinterpret_cast<uint32_t*>(dyn);
  int32_t* ahead = dyn + words;
  int32_t* sums = dyn + 2 * words;  // pages needed ahead of sequence b, saturating
  uint32_t* refused = reinterpret_cast<uint32_t*>(sums + p.num_seqs + 1);
  uint32_t* needing = refused + (p.num_seqs + 31) / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)ptx::cluster_rank();
  const int page0 = rank * words * 32;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // What sequence b needs, and whether it gets anything (if not: said by the first CTA).
  auto need_of = [&](int b, bool& ok) {
    const Want w = wants(p, b, rank == 0);
    ok = w.ok;
    int64_t need = ok && w.want > w.have ? w.want - w.have : 0;
    const int* row = p.table + (int64_t)b * p.t_s0;
    for (int j = w.first; ok && j < w.have && j < w.want; ++j) {
      const int page = row[(int64_t)j * p.t_s1];
      ok = (unsigned)page < (unsigned)p.num_pages;  // (no place may look like a mark)
      if (!ok && rank == 0) report(p, kPgBadTable);
      need += is_shared(p, page);
    }
    return ok ? need : 0;
  };
  // 1a: the bitmap, a warp a word (32 pages); the first words' loads are under way while
  // the first sequences' needs are found
  constexpr int kWarps = kPoolThreads / 32, kEarly = 4;
  auto refs_of = [&](int w) {
    const int page = page0 + 32 * w + lane;
    return w < words && page < p.num_pages ? p.refs[page] : 1;
  };
  int early[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) early[k] = refs_of(warp + kWarps * k);
  bool ok0 = false;
  const int64_t need0 = tid < p.num_seqs ? need_of(tid, ok0) : 0;
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const uint32_t bits = __ballot_sync(0xffffffffu, early[k] == 0);
    if (lane == 0 && warp + kWarps * k < words) map[warp + kWarps * k] = bits;
  }
#pragma unroll 4
  for (int w = warp + kWarps * kEarly; w < words; w += kWarps) {
    const uint32_t bits = __ballot_sync(0xffffffffu, refs_of(w) == 0);
    if (lane == 0) map[w] = bits;
  }
  __syncthreads();
  {
    int64_t running = 0;
    for (int w0 = 0; w0 < words; w0 += kPoolThreads) {
      const int w = w0 + tid;
      const int n = w < words ? __popc(map[w]) : 0;
      int64_t total;
      const int64_t inc = block_inclusive(n, scratch, &total);
      if (w < words) ahead[w] = (int)(running + inc - n);
      running += total;
    }
    if (tid == 0) s_free = (int)running;
  }
  // 1b: the sequences' needs
  {
    int64_t running = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kPoolThreads) {
      const int b = b0 + tid;
      int64_t need = need0;
      bool ok = ok0;
      if (b0 > 0) {
        ok = false;
        need = b < p.num_seqs ? need_of(b, ok) : 0;
      }
      const uint32_t no = __ballot_sync(0xffffffffu, !ok), some = __ballot_sync(0xffffffffu, need > 0);
      if (lane == 0 && b < p.num_seqs) {
        refused[b >> 5] = no;
        needing[b >> 5] = some;
      }
      int64_t total;
      const int64_t inc = block_inclusive(need, scratch, &total);
      if (b < p.num_seqs) sums[b + 1] = (int)(running + inc < INT32_MAX ? running + inc : INT32_MAX);
      running += total;
    }
    if (tid == 0) sums[0] = 0;
  }
  cluster_meet();
  // free pages ahead of each CTA's part, and all
  int base[kPoolCtas + 1];
  base[0] = 0;
#pragma unroll
  for (int k = 0; k < kPoolCtas; ++k)
    base[k + 1] = base[k] + ld_cluster(ptx::cluster_addr(ptx::smem_addr(&s_free), k));
  const int all = base[kPoolCtas];
  // sequences get their pages as long as the sums stay within the free ones: ranks below
  // `granted` are given out
  int granted = 0;
  {
    int lo = 0, hi = p.num_seqs;  // the last sum that fits
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sums[mid] <= all)
        lo = mid;
      else
        hi = mid - 1;
    }
    granted = sums[lo];
  }
  auto needs = [&](int b) { return ((needing[b >> 5] >> (b & 31)) & 1) != 0; };
  auto grants = [&](int b) { return !((refused[b >> 5] >> (b & 31)) & 1) && (sums[b + 1] <= all || !needs(b)); };
  // 2: marks
  for (int b = rank + kPoolCtas * tid; b < p.num_seqs; b += kPoolCtas * kPoolThreads) {
    if (!needs(b)) continue;
    if (!grants(b)) {
      report(p, kPgNoPages);
      continue;
    }
    const Want w = wants(p, b, false);
    int* row = p.table + (int64_t)b * p.t_s0;
    for (int j = w.first; j < w.have && j < w.want; ++j) {
      const int page = row[(int64_t)j * p.t_s1];
      if (is_shared(p, page)) row[(int64_t)j * p.t_s1] = ~page;
    }
  }
  cluster_meet();
  // 3a: growing rows
  int my_base = 0;
#pragma unroll
  for (int k = 0; k < kPoolCtas; ++k)
    if (k == rank) my_base = base[k];
  for (int w = warp; w < words && my_base + ahead[w] < granted; w += kPoolThreads / 32) {
    const uint32_t bits = map[w];
    const int at = my_base + ahead[w] + __popc(bits & ((1u << lane) - 1));  // this page's rank
    if (!((bits >> lane) & 1) || at >= granted) continue;
    const int page = page0 + 32 * w + lane;
    p.refs[page] = 1;
    int lo = 0, hi = p.num_seqs - 1;  // the sequence with sums[b] <= at < sums[b + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sums[mid + 1] > at)
        hi = mid;
      else
        lo = mid + 1;
    }
    const Want s = wants(p, lo, false);
    const int grow = s.want > s.have ? s.want - s.have : 0;
    const int k = at - sums[lo] - (sums[lo + 1] - sums[lo] - grow);  // behind its replaced pages
    if (k >= 0)
      p.table[(int64_t)lo * p.t_s0 + (int64_t)(s.have + k) * p.t_s1] = page;
    else if (at == sums[lo])
      p.dst[lo] = page;  // the first replaced one's, for 3b
  }
  cluster_meet();
  // 3b: marked places
  auto page_of_rank = [&](int at) {
    int cta = 0;
#pragma unroll
    for (int k = 1; k < kPoolCtas; ++k)
      if (at >= base[k]) cta = k;
    int from = 0;
#pragma unroll
    for (int k = 0; k < kPoolCtas; ++k)
      if (k == cta) from = base[k];
    at -= from;
    const uint32_t a = ptx::cluster_addr(ptx::smem_addr(ahead), cta);
    int lo = 0, hi = words - 1;  // the last word with ahead <= at
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (ld_cluster(a + 4 * mid) <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    uint32_t bits = (uint32_t)ld_cluster(ptx::cluster_addr(ptx::smem_addr(map), cta) + 4 * lo);
    for (int k = at - ld_cluster(a + 4 * lo); k > 0; --k) bits &= bits - 1;
    return (cta * words + lo) * 32 + __ffs((int)bits) - 1;
  };
  for (int b = rank + kPoolCtas * tid; b < p.num_seqs; b += kPoolCtas * kPoolThreads) {
    int src = -1, dst = -1;
    const Want w = wants(p, b, false);
    const bool ok = grants(b);
    if (ok && needs(b)) {
      const int first = __ldcg(p.dst + b);
      int* row = p.table + (int64_t)b * p.t_s0;
      int at = sums[b];
      for (int j = w.first; j < w.have && j < w.want; ++j) {
        const int mark = row[(int64_t)j * p.t_s1];
        if (mark >= 0) continue;
        const int page = at == sums[b] ? first : page_of_rank(at);
        ++at;
        row[(int64_t)j * p.t_s1] = page;
        atomicSub(p.refs + ~mark, 1);
        if (j == w.first && p.seqused[b] % kPageSize != 0) {  // it holds tokens
          src = ~mark;
          dst = page;
        }
      }
    }
    p.src[b] = src;
    p.dst[b] = dst;
    const int held = ok && w.want > w.have ? w.want : w.have;
    p.room[b] = (held < 0 ? 0 : held > p.width ? p.width : held) * kPageSize;
  }
  cluster_meet();  // (nobody reads the counts or another CTA's bitmap any more)
  // 4
  for (int b = rank + kPoolCtas * tid; b < p.num_seqs; b += kPoolCtas * kPoolThreads) {
    const Want w = wants(p, b, false);
    if (grants(b) && w.want > w.have) p.page_count[b] = w.want;
  }
}

cudaLaunchAttribute programmatic() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

}  // namespace

cudaError_t launch_copy_pages(const CopyParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)kPageSize * p.heads * p.units, per = kCopyThreads * kCopyUnits;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n, (unsigned)((units + per - 1) / per), p.c[1].data ? 2u : 1u);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {programmatic()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, va_copy_pages_kernel, p);
}

static cudaError_t launch_rows(void (*fn)(const PoolParams), const PoolParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n);
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1] = {programmatic()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

cudaError_t launch_free_pages(const PoolParams& p, cudaStream_t stream) { return launch_rows(va_free_pages_kernel, p, stream); }
cudaError_t launch_fork_pages(const PoolParams& p, cudaStream_t stream) { return launch_rows(va_fork_pages_kernel, p, stream); }

cudaError_t launch_reserve_pages(const PoolParams& p, cudaStream_t stream) {
  const int words = (p.num_pages + 32 * kPoolCtas - 1) / (32 * kPoolCtas);
  const size_t smem = sizeof(int32_t) * (2 * (size_t)words + (size_t)p.num_seqs + 1 + 2 * (((size_t)p.num_seqs + 31) / 32));
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(va_reserve_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPoolCtas);
  cfg.blockDim = dim3(kPoolThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {programmatic()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPoolCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, va_reserve_pages_kernel, p, words);
}

}  // namespace va
