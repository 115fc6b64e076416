// Attention of chunks of new tokens over the paged cache, on pairs of CTAs.
//
// Token t of a sequence of S cached tokens, L of them new, sees the keys up to S - L + t
// (with a window: those above S - L + t - W, and the first tokens), and
//   out = sum_j 2^(s_j - m) V_j / sum_j 2^(s_j - m),   s = log2(e) softmax_scale q . k_j,
// with soft cap and sinks as the verify kernels. One pass over the keys: O and the row's
// sum l are kept relative to a reference m that follows the running maximum, and are
// rescaled when a tile passes it by more than 2^8.
//
// The rows of a KV head are the G query heads of each token, packed: row = token G + head.
// An item is 256 rows of a sequence and KV head, 128 to each CTA of a pair (two SMs, one
// tcgen05 MMA of M = 256): each CTA brings half of every tile's keys and half of its values'
// columns, so a tile of 128 keys is read from L2 once for 256 rows and a CTA's shared memory
// holds the item's Q and two to four tiles of each kind. S and P share tensor memory
// (P is written over S); O takes 256 columns of it, two S buffers the other 256.
//
// Work is split by units (about keys times rows): every pair takes an equal run of them,
// found from closed forms, so a long prompt, a few tokens over a long cache and a ragged batch
// all fill the machine; an item that two pairs share leaves fp32 partials, which the merge
// kernel sums in the pairs' order (the same bits at every call). Few and short items have a
// pair each (kWholeTiles).
//
// What bounds it: 4 * 256 flops a visible (row, key) pair on the tensor cores; over long caches
// it runs there (2,048 tokens, 16 query heads over one KV head: bf16 over 63K keys 1.12 ms, 1.93
// PFLOP/s, e4m3 over 129K 2.35 ms, 1.86; the cuBLAS peak measured here is 1.91). At
// that rate a tile's MMAs take 1.3 us, in which each CTA's softmax has to be through with one
// too: 16 warps, in two groups that take the tiles in turn (e4m3 with 8 warps 2.87 ms,
// 2.45 when they became 16). Page scales cost the softmax a multiply
// and a sum for each page (1.62 ms, 1.34 PFLOP/s), the soft cap an exponential and a division a logit
// (1.86 ms, 1.16). Short calls are bound by the chain of share, Q, tiles and epilogue: two
// sequences of 25 and 21 tokens over 461 and 320 keys 19.0 us. One token in each of many sequences
// fills 16 of an item's 256 rows: 88-97 us for 269 MB, 2.8-3.1 TB/s.
//
// e4m3 caches: K's codes go to the MMA as they are (kind::f8f6f4), with Q as two e4m3 terms,
// which holds bf16's 8 bits at the rate of one bf16 product; V's codes become f16 on the way
// (exactly), for weights in f16.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "va_chunk.h"
#include "va_fp8.cuh"
#include "va_ptx.cuh"

namespace va {
namespace {

using namespace ptx;

constexpr int kKeys = kChunkKeys;
constexpr float kLog2e = 1.4426950408889634f;

// n / p.group for 0 <= n < 2^31: with s = ceil(log2 d) and m = floor(2^(31 + s) / d) + 1,
// n m / 2^(31 + s) is above n / d by less than 1 / d (0 < m d - 2^(31 + s) <= d <= 2^s).
__device__ __forceinline__ int by_group(const ChunkParams& p, int n) {
  return p.group == 1 ? n : (int)(__umulhi((uint32_t)n, p.group_m) >> p.group_s);
}

// ---- the split of the work ----------------------------------------------------------

struct Seq {
  int S, L, q0;  // cached tokens, new tokens, first row of q; clamped to the buffers
};

__device__ __forceinline__ Seq chunk_seq(const ChunkParams& p, int b) {
  const int a = p.cu_q[b], e = p.cu_q[b + 1];
  Seq s;
  s.q0 = a;
  s.L = a < 0 || e <= a ? 0 : e - a;
  const int room = p.total_q - a;
  if (s.L > room) s.L = room < 0 ? 0 : room;
  s.S = p.seqused_k[b];
  const int cap = p.num_blocks > 0 ? p.bt_width * kPageSize : 0;
  s.S = s.S < 0 ? 0 : s.S > cap ? cap : s.S;
  return s;
}

__device__ __forceinline__ int row_tiles(const ChunkParams& p, const Seq& s) {
  return (int)(((int64_t)s.L * p.group + kChunkRows - 1) / kChunkRows);
}

// Small calls. Where there are no more items than pairs, and none costs more than kWholeTiles
// tiles (its start among them), an item has a pair to itself and nothing is joined; else a share
// has at least kMinShare tiles, so that fewer pairs take part, whose partials cost more to
// write and to join than the tiles they save. us a call, geometric means over 24 to 30 random
// calls each: two sequences of 17-48 tokens over 200-1,024 keys (16 query heads over one)
// 22.3 whole, 26.7 / 27.2 / 29.7 in shares of at least 3 / 4 / 7 tiles (2: 26.6, 5: 28.0, 10:
// 29.8); up to three of 10-60 tokens over 900-3,500 keys 34.9 with items of up to 18 tiles
// whole (16: 35.0, 20: 35.2, 24: 35.6, 28: 38.2); one of 100-900 tokens over 900-1,500 keys
// 27.5 whole, 34.5 / 35.2 / 37.3 in shares of at least 3 / 4 / 7.
constexpr int64_t kWholeTiles = 18;
constexpr int64_t kMinShare = 3;

// Units of the split: a tile is 128 G of them. Row tile m costs
//   min(max(0, (S - L) G + 256 (m + 1)), cap) + kChunkItemCost * 128 G,
// about G times the keys that its rows see, so that the sum over a sequence's
// row tiles has a closed form and a share's start is found without walking them.
// The sum of tiles that an item really has (window and first tokens start and
// end inside tiles) is at most 3 above keys / 128.
__device__ __forceinline__ int64_t unit_cap(const ChunkParams& p) {
  if (p.window_left < 0) return INT64_MAX / 4;
  return ((int64_t)p.window_left + 2 + p.first_tokens) * p.group + kChunkRows;
}

__device__ __forceinline__ int64_t chunk_cost(const ChunkParams& p, const Seq& s, int m) {
  const int64_t x = (int64_t)(s.S - s.L) * p.group + (int64_t)kChunkRows * (m + 1);
  const int64_t cap = unit_cap(p);
  return (x < 0 ? 0 : x > cap ? cap : x) + (int64_t)kChunkItemCost * kKeys * p.group;
}

// Units of row tiles [0, m).
__device__ __forceinline__ int64_t chunk_prefix(const ChunkParams& p, const Seq& s, int64_t m) {
  const int64_t x0 = (int64_t)(s.S - s.L) * p.group, cap = unit_cap(p);
  int64_t a = x0 < 0 ? -x0 / kChunkRows : 0;           // tiles below a cost nothing but their start
  int64_t b = cap <= x0 ? 0 : (cap - x0) / kChunkRows;  // tiles from b on cost cap
  a = a > m ? m : a;
  b = b > m ? m : b < a ? a : b;
  return m * ((int64_t)kChunkItemCost * kKeys * p.group) + (b - a) * x0 + kChunkRows / 2 * (b * (b + 1) - a * (a + 1)) +
         (m > b ? (m - b) * cap : 0);
}

// The keys that an item's rows see: [0, khi), or with a window [klo, khi) and the
// first tokens; its tiles: nf from 0 on, then those from w0 on, n in all.
struct Span {
  int klo, khi, nf, w0, n;
};

__device__ __forceinline__ Span item_span(const ChunkParams& p, const Seq& s, int m) {
  const int row0 = kChunkRows * m;  // (rows fit an int)
  const int t0 = by_group(p, row0);
  int t1 = by_group(p, row0 + kChunkRows - 1);
  t1 = t1 < s.L - 1 ? t1 : s.L - 1;
  Span x;
  x.khi = s.S - s.L + t1 + 1;
  x.khi = x.khi < 0 ? 0 : x.khi;
  x.klo = 0;
  if (p.window_left >= 0) {
    const int64_t lo = (int64_t)s.S - s.L + t0 - p.window_left;
    x.klo = lo < 0 ? 0 : (int)lo;
  }
  x.w0 = x.klo / kKeys;
  x.nf = 0;
  if (p.window_left >= 0 && p.first_tokens > 0) {
    x.nf = (int)(((int64_t)p.first_tokens + kKeys - 1) / kKeys);
    x.nf = x.nf < x.w0 ? x.nf : x.w0;
  }
  x.n = x.khi > 0 ? x.nf + (x.khi - 1) / kKeys + 1 - x.w0 : 0;  // (khi itself may end 16 below 2^31)
  return x;
}

// 64-bit quotients, by a 32-bit division (a tenth of the instructions) where they fit.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
  return (uint64_t)x <= 0xFFFFFFFFu && (uint64_t)y <= 0xFFFFFFFFu ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// A share's units, and the first of share c's.
__device__ __forceinline__ int64_t share_units(int64_t total, int used) { return used > 0 ? quotient(total + used - 1, used) : 0; }
__device__ __forceinline__ int64_t share_begin(int64_t total, int64_t share, int c) {
  const int64_t t = share * c;
  return t < total ? t : total;
}

// Tiles of 128 G units that x units reach into.
__device__ __forceinline__ int64_t ceil_units(const ChunkParams& p, int64_t x) {
  if (x <= 0) return 0;
  const int64_t t = (x + kKeys - 1) / kKeys;  // in G
  return t + p.group <= 0x7FFFFFFF ? by_group(p, (int)(t + p.group - 1)) : (t + p.group - 1) / p.group;
}

// Walks the items from a share's start on.
struct Walk {
  int b, h, m, tiles;
  int64_t off;
  Seq s;
};

__device__ __forceinline__ Walk start_walk(const ChunkParams& p, const ChunkStart& st) {
  Walk w;
  w.b = st.b;
  w.h = st.h;
  w.m = st.m;
  w.off = st.off;
  w.s = chunk_seq(p, st.b);
  w.tiles = row_tiles(p, w.s);
  return w;
}

// An item's part in a share: tiles [i0, i0 + n) of the item's.
struct Piece {
  int n;                    // -1: no further piece
  int h, m, i0;
  int S, L, q0, b;
  Span x;
  int direct;               // the whole item: its rows are written to out
};

__device__ __forceinline__ bool next_piece(const ChunkParams& p, int64_t t0, int64_t t1, Walk& w, Piece& pc) {
  while (w.off < t1) {
    if (w.m >= w.tiles) {
      w.m = 0;
      if (w.tiles == 0 || ++w.h == p.hkv) {
        w.h = 0;
        if (++w.b >= p.num_seqs) return false;
        w.s = chunk_seq(p, w.b);
        w.tiles = row_tiles(p, w.s);
      }
      continue;
    }
    pc.b = w.b;
    pc.h = w.h;
    pc.m = w.m;
    pc.S = w.s.S;
    pc.L = w.s.L;
    pc.q0 = w.s.q0;
    pc.x = item_span(p, w.s, w.m);
    const int64_t off = w.off;
    w.off += chunk_cost(p, w.s, w.m);
    ++w.m;
    int64_t i0 = ceil_units(p, t0 - off), i1 = ceil_units(p, t1 - off);
    i0 = i0 < pc.x.n ? i0 : pc.x.n;
    i1 = i1 < pc.x.n ? i1 : pc.x.n;
    pc.i0 = (int)i0;
    pc.n = (int)(i1 - i0);
    pc.direct = i0 == 0 && i1 == pc.x.n;
    if (pc.n > 0 || (pc.x.n == 0 && off >= t0)) return true;
  }
  return false;
}

__device__ __forceinline__ int tile_of(const Span& x, int i) { return i < x.nf ? i : x.w0 + (i - x.nf); }

// ---- the main kernel -----------------------------------------------------------------

enum Kind { kBf16 = 0, kE4m3 = 1, kPageScaled = 2 };

constexpr int kSoftmaxWarps = 16;
constexpr int kPieces = 3;  // places of the queue of pieces
constexpr int kMiscSize = 3 * 1024;  // barriers and small arrays behind the tiles

// Shared memory: Q, then K's ring and V's. K goes to the MMAs as TMA brings it. So does a
// bf16 V; e4m3 codes of V become f16 on the way, from a ring of their own. A waiter meets
// every phase of its barriers: a ring has one producer, and a slot one user (e4m3 V:
// two slots for two groups, tile by tile in turn).
template <int KIND>
struct Cfg {
  static constexpr bool kFp8 = KIND != kBf16;
  // Warps: softmax, loaders (two groups of four, which convert e4m3 V in turn), two
  // producers, the MMA's and the planner. Registers a thread: each warpgroup trades its
  // share of the launch's 72; the last one, with the MMA issuer, is the one that pays
  // most for a spill (80 / 56 / 56: bf16 1,190 us where this takes 1,138).
  static constexpr int kLoadGroups = 2, kLoadWarps = 4 * kLoadGroups;
  static constexpr int kWarpProducer = kSoftmaxWarps + kLoadWarps, kWarpMma = kWarpProducer + 2, kWarpPlan = kWarpMma + 1;
  static constexpr int kThreads = 32 * (kWarpPlan + 1);
  static constexpr int kLaunchRegs = 72, kSoftmaxRegs = 80, kLoadRegs = 48, kOtherRegs = 88;
  static_assert(4 * kSoftmaxRegs + kLoadGroups * kLoadRegs + kOtherRegs <= (5 + kLoadGroups) * kLaunchRegs, "registers");
  static_assert(kThreads * kLaunchRegs <= 65536, "registers");
  static constexpr int kKBytes = kFp8 ? 16384 : 32768;  // a CTA's half of a K tile: 64 keys
  static constexpr int kVBytes = 32768;                 // .. of a V tile, 16 bits: 128 columns
  static constexpr int kRawBytes = 16384;               // .. as e4m3
  static constexpr int kKSlots = kFp8 ? 4 : 2, kVSlots = kFp8 ? 2 : 3, kRawSlots = kFp8 ? 2 : 0;
  static constexpr int kOffQ = 0;  // [4][128 rows][128 bytes]: d chunks (bf16), or two of each e4m3 term
  static constexpr int kOffK = 65536;
  static constexpr int kOffV = kOffK + kKSlots * kKBytes;
  static constexpr int kOffRaw = kOffV + kVSlots * kVBytes;
  static constexpr int kOffMisc = kOffRaw + kRawSlots * kRawBytes;
  static constexpr int kSmemBytes = kOffMisc + kMiscSize;
  static_assert(kSmemBytes <= 232448, "shared memory");
  // what TMA fills: V's own ring, or the codes'
  static constexpr int kTmaVSlots = kFp8 ? kRawSlots : kVSlots;
  static constexpr int kTmaVBytes = kFp8 ? kRawBytes : kVBytes, kOffTmaV = kFp8 ? kOffRaw : kOffV;
  // instruction descriptors, M = 256: bf16 (1) or e4m3 (0), and f16 (0)
  static constexpr uint32_t kIdQK = instr_desc(kFp8 ? 0u : 1u, kFp8 ? 0u : 1u, false, kKeys, 256);
  static constexpr uint32_t kIdPV = instr_desc(kFp8 ? 0u : 1u, kFp8 ? 0u : 1u, true, kHeadDim, 256);
};

// misc area: barriers, pieces, row factors, page scales
constexpr int kMaxK = 4, kMaxV = 3;
// Tiles whose page scales are kept: the producer, up to four K tiles ahead of the MMAs,
// writes tile i's once the softmax is through with tile i - 6.
constexpr int kScaleTiles = 6;
enum : int {
  kBarKFull = 0,                      // this CTA's half has landed
  kBarKPeer = kBarKFull + kMaxK,      // .. the odd CTA's (in the even one)
  kBarKEmpty = kBarKPeer + kMaxK,
  kBarVLanded = kBarKEmpty + kMaxK,   // what TMA brought of V
  kBarRawEmpty = kBarVLanded + kMaxV,  // e4m3: converted
  kBarVFull = kBarRawEmpty + 2,       // V as the MMAs take it, both CTAs' halves
  kBarVEmpty = kBarVFull + kMaxV,
  kBarSFull = kBarVEmpty + kMaxV,
  kBarPFull = kBarSFull + 2,
  kBarPvDone = kBarPFull + 2,
  kBarQFull = kBarPvDone + 2,
  kBarQFree,
  kBarOFree,
  kBarDrain,
  kBarScales,
  kBarPieceFull = kBarScales + kScaleTiles,
  kBarPieceEmpty = kBarPieceFull + kPieces,
  kNumBars = kBarPieceEmpty + kPieces
};
constexpr int kOffTmem = 8 * kNumBars, kOffAbort = kOffTmem + 4;
constexpr int kOffIssued = kOffAbort + 4;  // K tiles and V tiles that TMA has been told to bring
// ChunkStart, in bytes of its own: it is read (for the merge, by the planner) while the
// planner writes pieces already
constexpr int kOffStart = (kOffIssued + 8 + 15) / 16 * 16;
constexpr int kOffPieces = kOffStart + (sizeof(ChunkStart) + 15) / 16 * 16;  // [kPieces] Piece
constexpr int kOffRow = kOffPieces + kPieces * 64;               // [2][128] exponents of Q's rows (bytes)
constexpr int kOffXch = kOffRow + 256;                           // [2][128] floats; before: 32 x 8 bytes of the scan
constexpr int kOffRef = kOffXch + 1024;                          // [128] floats: the rows' references
constexpr int kOffScale = kOffRef + 512;                         // [kScaleTiles][8] (K scale, log2 V scale)
constexpr int kMiscBytes = kOffScale + kScaleTiles * 64;
static_assert(kMiscBytes <= kMiscSize && sizeof(Piece) <= 64, "misc area");
static_assert(kOffStart + sizeof(ChunkStart) <= kOffPieces, "nothing lies over the start");

constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;

// P = 2^(s - m_ref + shift): m_ref moves when a tile's max passes it by more than
// kMove (O and l are rescaled then). bf16 keeps 8 bits at any size; f16 holds up to
// 2^15 with shift 7 and all its 11 bits down to 2^-21 of 2^m_ref.
constexpr float kMove = 8.f;

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// VAR: with the code of the window and the soft cap.
template <int KIND, bool VAR>
__global__ void __launch_bounds__(Cfg<KIND>::kThreads, 1)
    va_chunk_kernel(const ChunkParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  using C = Cfg<KIND>;
  constexpr bool kFp8 = C::kFp8;
  constexpr bool kScl = KIND == kPageScaled;
  constexpr int kThreads = C::kThreads, kLoadWarps = C::kLoadWarps;
  constexpr int kWarpProducer = C::kWarpProducer, kWarpMma = C::kWarpMma, kWarpPlan = C::kWarpPlan;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = smem_raw;
  unsigned char* misc = sm + C::kOffMisc;
  const uint32_t sbase = smem_addr(sm);
  const uint32_t mbase = sbase + C::kOffMisc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + kOffAbort);
  long long* scratch = reinterpret_cast<long long*>(misc + kOffXch);
  ChunkStart* start = reinterpret_cast<ChunkStart*>(misc + kOffStart);
  volatile int* issued = reinterpret_cast<volatile int*>(misc + kOffIssued);
  unsigned char* row_exp = misc + kOffRow;
  float* refs = reinterpret_cast<float*>(misc + kOffRef);
  float* xch = reinterpret_cast<float*>(misc + kOffXch);
  float2* page_scale = reinterpret_cast<float2*>(misc + kOffScale);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank();
  const int c = blockIdx.x >> 1;
  auto bar = [&](int i) { return mbase + 8 * i; };
  auto lead = [&](int i) { return cluster_addr(mbase + 8 * i, 0); };  // the issuing CTA's barrier

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < C::kKSlots; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarKPeer + i), 1);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < C::kTmaVSlots; ++i) mbar_init(bar(kBarVLanded + i), 1);
    for (int i = 0; i < C::kRawSlots; ++i) mbar_init(bar(kBarRawEmpty + i), 4);
    for (int i = 0; i < C::kVSlots; ++i) {
      mbar_init(bar(kBarVFull + i), kFp8 ? 2 * 4 : 2);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), kSoftmaxWarps);  // a group's eight warps of each CTA
      mbar_init(bar(kBarPvDone + i), 1);
    }
    mbar_init(bar(kBarQFull), 2 * kLoadWarps);
    mbar_init(bar(kBarQFree), 1);
    mbar_init(bar(kBarOFree), 2 * kSoftmaxWarps);
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < kScaleTiles; ++i) mbar_init(bar(kBarScales + i), 1);
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bar(kBarPieceFull + i), 1);
      mbar_init(bar(kBarPieceEmpty + i), kWarpPlan);  // every warp before it
    }
    *abort_flag = 0;
    issued[0] = issued[1] = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(mbase + kOffTmem, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == kWarpProducer && lane == 0 && p.num_blocks > 0) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // barriers are set up before the other CTA arrives on them
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(misc + kOffTmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- this pair's share
  int64_t t0 = 0, t1 = 0;
  {
    const int64_t unit = (int64_t)kKeys * p.group;
    int64_t total = 0, mine = 0, ex = 0;
    Seq s{};
    if (p.num_seqs <= kThreads) {
      if (tid < p.num_seqs) {
        s = chunk_seq(p, tid);
        mine = p.hkv * chunk_prefix(p, s, row_tiles(p, s));
      }
      long long tot;
      ex = block_exclusive_scan<kThreads>(mine, scratch, &tot);
      total = tot;
    } else {
      for (int b0 = 0; b0 < p.num_seqs; b0 += kThreads) {
        int64_t v = 0;
        if (b0 + tid < p.num_seqs) {
          const Seq q = chunk_seq(p, b0 + tid);
          v = p.hkv * chunk_prefix(p, q, row_tiles(p, q));
        }
        long long tot;
        block_exclusive_scan<kThreads>(v, scratch, &tot);
        total += tot;
      }
    }
    bool whole = false;
    if (p.force <= 0 && p.num_seqs <= kThreads && total > 0 && total <= kWholeTiles * unit * p.pairs) {
      const int tiles = tid < p.num_seqs ? row_tiles(p, s) : 0;  // (the last of them costs most)
      if (!__syncthreads_or(tiles > 0 && chunk_cost(p, s, tiles - 1) > kWholeTiles * unit)) {
        const int64_t items = (int64_t)tiles * p.hkv;
        long long all;
        const int64_t first = block_exclusive_scan<kThreads>(items, scratch, &all);
        whole = all <= p.pairs;
        if (whole && c < all) {  // pair c takes item c; its units are counted from the item's first
          if (first <= c && c < first + items) {
            start->b = tid;
            start->h = (c - (int)first) / tiles;
            start->m = (c - (int)first) % tiles;
            start->off = 0;
            start->total = chunk_cost(p, s, start->m);
          }
          __syncthreads();
          t1 = start->total;
        }
      }
    }
    // as many pairs as get at least kMinShare tiles' units each
    int used = p.force > 0 && p.force < p.pairs ? p.force : p.pairs;
    if (p.force <= 0 && total < kMinShare * unit * p.pairs) used = (int)quotient(total, kMinShare * unit);
    used = total == 0 || whole ? 0 : used < 1 ? 1 : used;
    const int64_t share = share_units(total, used);
    // The rounding up can leave the last pairs nothing: they are not counted, so that each
    // counted share has a first unit and an item that it starts in. The share of the smaller
    // count is the same: it is at least ceil(total / used), and share * count >= total.
    if (share > 0) used = (int)quotient(total + share - 1, share);
    if (c < used) {
      t0 = share_begin(total, share, c);
      t1 = share_begin(total, share, c + 1);
      int64_t running = 0;
      for (int b0 = 0; b0 < p.num_seqs; b0 += kThreads) {
        if (p.num_seqs > kThreads) {
          mine = 0;
          if (b0 + tid < p.num_seqs) {
            s = chunk_seq(p, b0 + tid);
            mine = p.hkv * chunk_prefix(p, s, row_tiles(p, s));
          }
          long long tot;
          ex = block_exclusive_scan<kThreads>(mine, scratch, &tot);
          ex += running;
          running += tot;
        }
        if (mine > 0 && ex <= t0 && t0 < ex + mine) {
          const int tiles = row_tiles(p, s);
          const int64_t per = chunk_prefix(p, s, tiles);
          const int64_t h = quotient(t0 - ex, per), at = t0 - ex - h * per;
          int lo = 0, hi = tiles;  // the largest m with prefix(m) <= at
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_prefix(p, s, mid) <= at)
              lo = mid;
            else
              hi = mid;
          }
          start->b = b0 + tid;
          start->h = (int)h;
          start->m = lo;
          start->off = ex + h * per + chunk_prefix(p, s, lo);
          start->total = total;
          start->used = used;
        }
      }
      __syncthreads();
      if (tid == 0 && rank == 0) p.ws_start[c] = *start;
    } else if (c == 0 && tid == 0 && rank == 0) {
      p.ws_start[0].used = 0;
    }
  }
  __syncwarp();
  cluster_wait();

  auto give_up = [&](int code) {
    *abort_flag = 1;
    st_cluster_u32(cluster_addr(mbase + kOffAbort, (uint32_t)(rank ^ 1)), 1u);
    if (p.ws_status) atomicOr(p.ws_status, code);
  };
  // Waits of a whole warp: warp-uniform, false once anything has given up.
  bool ok = true;
  auto wait_for = [&](int b, int use, int code) {
    if (!ok) return false;
    if (!__all_sync(0xffffffffu, mbar_wait(bar(b), (uint32_t)use & 1u, abort_flag, p.wait_limit_ns))) {
      if (lane == 0) give_up(code);
      ok = false;
    }
    return ok;
  };

  if (t0 < t1) {
    // The pieces of the share, walked by one warp for all roles. A role's warp takes the
    // next one (`at` counts them) and gives it back when it is through with it.
    volatile Piece* pieces = reinterpret_cast<volatile Piece*>(misc + kOffPieces);
    int at = 0;
    auto take = [&]() -> const volatile Piece* {
      const volatile Piece* pc = pieces + at % kPieces;
      return wait_for(kBarPieceFull + at % kPieces, at / kPieces, 8192) && pc->n >= 0 ? pc : nullptr;
    };
    auto give_back = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarPieceEmpty + at % kPieces));
      ++at;
    };
    if (warp < kSoftmaxWarps) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
      // ======================= softmax / epilogue =====================================
      // Two groups of eight warps: group 0 takes the tiles in S buffer 0, group 1 those in
      // buffer 1, so that one tile's chain of latencies (load, maximum, powers, store) runs
      // beside the next one's. Two warps of a group share a lane quadrant, a thread one
      // row and 64 keys. A row's reference goes from tile to tile, and so from group to
      // group, as soon as the tile's maximum is known; l stays with the thread. In the
      // epilogue a warp writes a quarter of O's columns. After a failure a warp walks on
      // without waits and work, so that they still meet at every named barrier (1 + q: a
      // group's two warps, whose turn the reference's way grants; 5 + q and 9 + q: that way
      // to group 0 and to group 1; 13: all). They want whole warps, as TMEM loads do: a warp
      // whose lanes took different ways (row_ok, a lane's arrival) is brought together first.
      const int q = warp & 3, kh = (warp >> 2) & 1, grp = warp >> 3;
      const uint32_t lane_base = (uint32_t)(32 * q) << 16;
      const int r = 32 * q + lane;  // this CTA's row
      const float kd = p.k_descale ? *p.k_descale : 1.f;
      const float cscale = fmaxf(fabsf(p.scale_log2 * kd), 1e-30f);  // the sign is Q's
      constexpr float kShift = kFp8 ? 7.f : 0.f;
      int tiles = 0, piece = 0;
      while (true) {
        const volatile Piece* pc = take();
        __syncwarp();
        if (named_bar_or(13, 32 * kSoftmaxWarps, pc == nullptr)) break;  // (all leave together)
        const int n = pc->n;
        const int row0 = pc->m * kChunkRows + rank * 128;  // this CTA's first row
        const bool idle = row0 + 32 * q >= pc->L * p.group;  // no row of the quadrant's
        const int t_r = by_group(p, row0 + r);  // the row's token
        // keys that this row sees: up to vis_end, from vis_lo on or below first_tokens;
        // tiles with keys past end_min, or before lo_max, are masked
        const int vis_end = t_r < pc->L ? pc->S - pc->L + t_r : -1;
        const int end_min = pc->S - pc->L + by_group(p, pc->m * kChunkRows);
        int vis_lo = 0, lo_max = 0;
        if (VAR && p.window_left >= 0) {
          const int64_t lo = (int64_t)vis_end - p.window_left, hi = (int64_t)pc->x.khi - 1 - p.window_left;
          vis_lo = lo < 0 ? 0 : (int)lo;
          lo_max = hi < 0 ? 0 : (int)hi;
        }
        const int tile0 = pc->i0;
        const int jump = VAR ? pc->x.nf : 0, jump_to = VAR ? pc->x.w0 : 0;
        float m_ref = -INFINITY, l = 0.f, rs = cscale;
        bool first = true;  // of this group's tiles
        for (int i = (tiles & 1) ^ grp; i < n; i += 2) {
          const int cur = tiles + i;
          if (kScl) wait_for(kBarScales + cur % kScaleTiles, cur / kScaleTiles, 512);
          wait_for(kBarSFull + grp, cur >> 1, 256);
          __syncwarp();  // (a lane reports a wait that runs out)
          tc_fence_after();
          const uint32_t ts = tmem + lane_base + kColS + grp * kKeys + 64 * kh;  // this warp's keys
          const int tile = tile0 + i;
          const int key0 = (VAR && tile >= jump ? tile - jump + jump_to : tile) * kKeys + 64 * kh;
          const bool mask_hi = key0 + 63 > end_min, mask_lo = VAR && key0 < lo_max;
          const float2* scales = page_scale + (cur % kScaleTiles) * 8 + 4 * kh;
          const bool cap = VAR && p.softcap_log2 > 0.f;
          // S is read twice, 32 keys at a time: for the row's maximum and for P (its 128
          // values would leave a thread no registers, and half the block no threads; a
          // read takes 100 cycles)
          auto load = [&](int part, uint32_t (&x)[32]) {
            tmem_ld_32x32b_x32(ts + 32 * part, x);
            tmem_wait_ld();
          };
          constexpr uint32_t kHidden = 0xFF800000u;  // -inf
          auto mask = [&](int part, uint32_t (&x)[32]) {
            if (mask_hi) {
              const int end = vis_end - key0 - 32 * part;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k > end) x[k] = kHidden;
            }
            if (mask_lo) {
              const int lo = vis_lo - key0 - 32 * part, keep = p.first_tokens - key0 - 32 * part;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (k < lo && k >= keep) x[k] = kHidden;
            }
          };
          // a key's logit (log2 units) is x times this; positive and normal, so that a masked
          // key's -inf stays that
          auto factor = [&](float ks) { return cap ? p.softcap_log2 : fmaxf(rs * ks, 1.2e-38f); };
          float top = -INFINITY;
          if (ok && !idle) {
            if (kFp8 && first) rs = fmaxf(cscale * __uint_as_float((uint32_t)row_exp[(piece & 1) * 128 + r] << 23), 1.2e-38f);
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t x[32];
              load(part, x);
              if (cap) {
                // c tanh(s / c) = c (1 - 2 / (e^(2 s / c) + 1)), kept without the factor c
                // in S's place
                const float f = rs * ((2.f * kLog2e) / p.softcap_log2);
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  const float y = __uint_as_float(x[k]) * (kScl ? f * scales[2 * part + k / kPageSize].x : f);
                  x[k] = __float_as_uint(1.f - __fdividef(2.f, ex2(y) + 1.f));
                }
                tmem_st_32x32b_x32(ts + 32 * part, x);
              }
              mask(part, x);
              float u[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int k = 0; k < 32; k += 2)
                u[k / kPageSize] = fmax3(u[k / kPageSize], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
              if constexpr (kScl) {
                const float4 sc = *reinterpret_cast<const float4*>(scales + 2 * part);
                top = fmax3(top, fmaf(u[0], factor(sc.x), sc.y), fmaf(u[1], factor(sc.z), sc.w));
              } else {
                top = fmax3(top, u[0], u[1]);
              }
            }
            if (!kScl) top *= factor(1.f);
            if (cap) tmem_wait_st();
          }
          // the reference of the tile before, the other group's; the maximum of the row's
          // other keys
          float m_old = -INFINITY;
          if (i > 0) {
            named_bar(5 + 4 * grp + q, 128);
            m_old = refs[r];
          }
          xch[128 * kh + r] = top;
          named_bar(1 + q, 64);
          top = fmaxf(top, xch[128 * (kh ^ 1) + r]);
          const float m_new = top > m_old + kMove ? top : m_old;
          if (i + 1 < n) {
            if (kh == 0) refs[r] = m_new;
            named_arrive(5 + 4 * (grp ^ 1) + q, 128);
          }
          if (ok && !idle) {
            if (m_new != m_ref) {
              if (m_ref != -INFINITY) l *= ex2(m_ref - m_new);
              m_ref = m_new;
            }
            const bool move = m_new != m_old && m_old != -INFINITY;
            if (__any_sync(0xffffffffu, move)) {
              const float alpha = move ? ex2(m_old - m_new) : 1.f;
              // O holds earlier tiles (of this piece: m_old is not -inf)
              const bool settled = wait_for(kBarPvDone + (grp ^ 1), (cur - 1) >> 1, 2048);
              tc_fence_after();
              __syncwarp();
#pragma unroll 1
              for (int j = 0; settled && j < kHeadDim / 64; ++j) {
                uint32_t o[32];
                const uint32_t ta = tmem + lane_base + kColO + 128 * kh + 32 * j;
                tmem_ld_32x32b_x32(ta, o);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
                tmem_st_32x32b_x32(ta, o);
              }
            }
            // (a row without a visible key yet: P = 0)
            const float ref = m_ref == -INFINITY ? INFINITY : m_ref - kShift;
            uint64_t ls[2] = {0, 0};
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              uint32_t x[32], pw[16];
              load(part, x);
              mask(part, x);
              const float4 sc = kScl ? *reinterpret_cast<const float4*>(scales + 2 * part) : make_float4(1.f, 0.f, 1.f, 0.f);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float f = factor(k < 8 ? sc.x : sc.z), off = (k < 8 ? sc.y : sc.w) - ref;
                float a, d;
                unpack2(fma2(pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), pack2(f, f), pack2(off, off)), a, d);
                a = ex2(a);
                d = ex2(d);
                ls[k & 1] = add2(ls[k & 1], pack2(a, d));
                pw[k] = kFp8 ? pack_f16x2(a, d) : pack_b16x2(a, d);
                if (kScl && k % 8 == 7) {  // a page's end: its weights without the V scale
                  float s0, s1, s2, s3;
                  unpack2(ls[0], s0, s1);
                  unpack2(ls[1], s2, s3);
                  l = fmaf((s0 + s1) + (s2 + s3), ex2(-(k < 8 ? sc.y : sc.w)), l);
                  ls[0] = ls[1] = 0;
                }
              }
              // over S: this thread has loaded the columns
              tmem_st_32x32b_x16(ts + 16 * part, pw);
            }
            if (!kScl) {
              float s0, s1, s2, s3;
              unpack2(ls[0], s0, s1);
              unpack2(ls[1], s2, s3);
              l += (s0 + s1) + (s2 + s3);
            }
            tmem_wait_st();
          }
          first = false;
          if (ok) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(lead(kBarPFull + grp));
          }
        }
        // -- epilogue: the groups' references (O's is the larger) and the four sums
        tiles += n;
        __syncwarp();
        named_bar(13, 32 * kSoftmaxWarps);
        if (kh == 0) xch[128 * grp + r] = m_ref;
        named_bar(13, 32 * kSoftmaxWarps);
        const float m_row = fmaxf(xch[r], xch[128 + r]);
        if (m_ref != m_row) l = m_ref == -INFINITY ? 0.f : l * ex2(m_ref - m_row);
        m_ref = m_row;
        __syncwarp();
        named_bar(13, 32 * kSoftmaxWarps);
        if (kh == 1) xch[128 * grp + r] = l;
        named_bar(13, 32 * kSoftmaxWarps);
        if (kh == 0) xch[128 * grp + r] = l + xch[128 * grp + r];
        named_bar(13, 32 * kSoftmaxWarps);
        l = xch[r] + xch[128 + r];
        if (n > 0) {
          wait_for(kBarPvDone + ((tiles - 1) & 1), (tiles - 1) >> 1, 4096);
          tc_fence_after();
        }
        const bool row_ok = row0 + r < pc->L * p.group, direct = pc->direct;
        const int g = row0 + r - t_r * p.group, head = pc->h * p.group + g;
        const int64_t slot = 2 * (int64_t)c + (pc->i0 == 0 ? 1 : 0);
        uint16_t* dst = p.out + (int64_t)(pc->q0 + t_r) * p.o_s0 + (int64_t)head * p.o_s1 + 128 * grp + 64 * kh;
        give_back();  // (ahead of the stores, which an arrival would wait for)
        if (ok) {
          if (p.sinks && direct && row_ok && m_ref != -INFINITY) l += ex2(p.sinks[head] * kLog2e - (m_ref - kShift));
          const float vd = p.v_descale ? *p.v_descale : 1.f;
          const float inv = l > 0.f || l != l ? vd / l : 0.f;
          const bool nothing = m_ref == -INFINITY && l == l;  // (all of them NaN: NaN)
          const int64_t acc_row = slot * kChunkRows + rank * 128 + r;
          float* acc = p.ws_acc + acc_row * kHeadDim + 128 * grp + 64 * kh;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t o[32];
            __syncwarp();  // (rows behind the last one left the stores out)
            if (n > 0 && !idle) {
              tmem_ld_32x32b_x32(tmem + lane_base + kColO + 128 * grp + 64 * kh + 32 * j, o);
              tmem_wait_ld();
            }
            if (n > 0 && j == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_relaxed(lead(kBarOFree));
            }
            if (!row_ok) continue;
            if (direct) {
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[k] = nothing ? 0u : pack_b16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
              if (p.out_v8) {
                st_global_v8(dst + 32 * j, v);
                st_global_v8(dst + 32 * j + 16, v + 8);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  reinterpret_cast<uint4*>(dst + 32 * j)[k] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) st_global_v8(acc + 32 * j + 8 * k, o + 8 * k);
            }
          }
          if (!direct && row_ok && grp == 0 && kh == 0)
            *reinterpret_cast<float2*>(p.ws_ml + acc_row * 2) =
                make_float2(nothing ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref - kShift, l);
        }
        if (n > 0) ++piece;
      }
    } else if (warp < kSoftmaxWarps + kLoadWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoadRegs));
      // ======================= loaders ================================================
      // Q of an item, and V's tiles on their way from TMA to the MMAs: e4m3 codes become
      // f16 (exactly), rows past the last key that a row of the item sees become zeros (0
      // times what a slot behind the sequence's last token holds would reach O).
      const int lw = warp - kSoftmaxWarps;  // rows of Q
      const int lg = lw >> 2, lq = lw & 3;  // group, and warp of it
      const float kd = p.k_descale ? *p.k_descale : 1.f;
      const bool neg = p.scale_log2 * kd < 0.f;
      int piece = 0, tiles = 0;
      while (const volatile Piece* pc = take()) {
        const int n = pc->n, i0 = pc->i0, h = pc->h, m = pc->m, L = pc->L, q0 = pc->q0;
        const Span x{pc->x.klo, pc->x.khi, pc->x.nf, pc->x.w0, 0};
        give_back();
        if (n == 0) continue;
        if (piece > 0 && !wait_for(kBarQFree, piece - 1, 32)) break;
        // Q: rows lw, lw + 8, .. of this CTA's 128
        const int rows = L * p.group, row0 = m * kChunkRows + rank * 128;
        auto q_row = [&](int r) {  // this lane's eight columns of row r
          const int t = by_group(p, row0 + r), g = row0 + r - t * p.group;
          return p.q + (int64_t)(q0 + t) * p.q_s0 + (int64_t)(h * p.group + g) * p.q_s1 + 8 * lane;
        };
        if constexpr (!kFp8) {
          // straight into place, all rows under way at once; rows behind the last are zeros
          auto place = [&](int r) { return C::kOffQ + (lane >> 3) * (128 * 128) + r * 128 + (((lane & 7) ^ (r & 7)) << 4); };
#pragma unroll 4
          for (int r = lw; r < 128; r += kLoadWarps) {
            const bool on = row0 + r < rows;
            cp_async_16(sbase + place(r), on ? q_row(r) : p.q, on);
          }
          cp_async_wait_all();
          if (neg) {
#pragma unroll 1
            for (int r = lw; r < 128; r += kLoadWarps) {
              uint4* v = reinterpret_cast<uint4*>(sm + place(r));
              *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
            }
          }
        } else {
          // as two e4m3 terms of q times a power of two that brings the row's largest into
          // [2^7, 2^8): bf16's 8 bits, in steps of at most 2^-16 of the largest. Four rows at a
          // time.
#pragma unroll 1
          for (int r0 = lw; r0 < 128; r0 += 4 * kLoadWarps) {
            uint4 raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = r0 + kLoadWarps * k;
              raw[k] = row0 + r < rows ? *reinterpret_cast<const uint4*>(q_row(r)) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = r0 + kLoadWarps * k;
              const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
              float mx = 0.f;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xFFFF0000u))));
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              int e = 0;
              if (mx > 0.f && mx < INFINITY) {
                e = 7 - ((int)(__float_as_uint(mx) >> 23) - 127);
                e = e > 120 ? 120 : e < -120 ? -120 : e;
              }
              const float up = __uint_as_float((uint32_t)(e + 127) << 23) * (neg ? -1.f : 1.f);
              uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float a = __uint_as_float(w[j] << 16) * up, d = __uint_as_float(w[j] & 0xFFFF0000u) * up;
                const uint32_t h8 = pack_fp8x2(a, d);
                const float2 f = unpack_fp8x2(h8);
                hi[j >> 1] |= h8 << (16 * (j & 1));
                lo[j >> 1] |= pack_fp8x2(a - f.x, d - f.y) << (16 * (j & 1));
              }
              if (lane == 0) row_exp[(piece & 1) * 128 + r] = (unsigned char)(127 - e);
              unsigned char* to = sm + C::kOffQ + (lane >> 4) * (128 * 128) + r * 128 + ((((lane >> 1) & 7) ^ (r & 7)) << 4) + 8 * (lane & 1);
              *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
              *reinterpret_cast<uint2*>(to + 2 * 128 * 128) = make_uint2(lo[0], lo[1]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(lead(kBarQFull));
        ++piece;
        if (!kFp8 && lw > 0) continue;  // one warp hands the tiles on
        for (int i = 0; i < n && ok; ++i) {
          const int cur = tiles + i;
          if (kFp8 && (cur & 1) != lg) continue;
          // rows of V from this one on are seen by no row
          const int valid = x.khi - tile_of(x, i0 + i) * kKeys;
          if constexpr (kFp8) {
            if (!wait_for(kBarVLanded + lg, cur >> 1, 64)) break;
            if (cur > 1 && !wait_for(kBarVEmpty + lg, (cur >> 1) - 1, 128)) break;
            const unsigned char* raw = sm + C::kOffRaw + lg * C::kRawBytes;
            unsigned char* op = sm + C::kOffV + lg * C::kVBytes;
            const int u = lane & 7;
            // 16 codes a thread and step: unit u (16 columns) of a row
#pragma unroll 1
            for (int k0 = 0; k0 < 8; k0 += 2) {
              uint4 in8[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int row = (k0 + k) * 16 + lq * 4 + (lane >> 3);
                in8[k] = *reinterpret_cast<const uint4*>(raw + row * 128 + ((u ^ (row & 7)) << 4));
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int row = (k0 + k) * 16 + lq * 4 + (lane >> 3);
                const uint32_t in[4] = {in8[k].x, in8[k].y, in8[k].z, in8[k].w};
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const __half2_raw v = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(in[j >> 1] >> (16 * (j & 1))), __NV_E4M3);
                  h[j] = row < valid ? (uint32_t)v.x | ((uint32_t)v.y << 16) : 0u;
                }
                const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                unsigned char* dst = op + (u >> 2) * (128 * 128) + row * 128;
                // the lanes of the upper 64 columns write their second unit first: a row's
                // eight lanes then reach eight different units
                const int first = u >> 2;
                *reinterpret_cast<uint4*>(dst + (((2 * (u & 3) + first) ^ (row & 7)) << 4)) = first ? hi : lo;
                *reinterpret_cast<uint4*>(dst + (((2 * (u & 3) + (first ^ 1)) ^ (row & 7)) << 4)) = first ? lo : hi;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kBarRawEmpty + lg));
              mbar_arrive_cluster(lead(kBarVFull + lg));
            }
          } else {
            const int slot = cur % C::kVSlots;
            if (!wait_for(kBarVLanded + slot, cur / C::kVSlots, 64)) break;
            if (valid < kKeys) {
              unsigned char* op = sm + C::kOffV + slot * C::kVBytes;
              for (int k = (valid < 0 ? 0 : valid) * 16 + lane; k < kKeys * 16; k += 32)
                *reinterpret_cast<uint4*>(op + (k & 15) / 8 * (128 * 128) + (k >> 4) * 128 + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
              __syncwarp();
            }
            if (lane == 0) mbar_arrive_cluster(lead(kBarVFull + slot));
          }
        }
        tiles += n;
        if (!ok) break;
      }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
      if (warp == kWarpPlan) {
        Walk w = start_walk(p, *start);
        Piece pc;
        for (bool more = true; more && ok; ++at) {
          more = next_piece(p, t0, t1, w, pc);
          if (!more) pc.n = -1;
          if (at >= kPieces && !wait_for(kBarPieceEmpty + at % kPieces, at / kPieces - 1, 16384)) break;
          if (lane == 0) *reinterpret_cast<Piece*>(misc + kOffPieces + at % kPieces * sizeof(Piece)) = pc;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarPieceFull + at % kPieces));
        }
      } else if (warp < kWarpMma) {
        // ======================= TMA producers =========================================
        // One warp for K's tiles, one for V's. One 2 KB box (a page's 16 tokens x 128
        // bytes) a lane: this CTA's half of K's keys, or of V's columns. Pages that no row of
        // the item sees are not mapped perhaps: they are read past the cache's last page,
        // which TMA fills with zeros. Page ids are loaded two tiles ahead.
        const bool is_k = warp == kWarpProducer;
        constexpr int kDim = kFp8 ? 2 : 4;    // 128-byte chunks of a row
        constexpr int kEl = kFp8 ? 128 : 64;  // elements of a chunk
        const int chunks = is_k ? kDim : kDim / 2;
        const int box_page = lane / chunks + (is_k ? 4 * rank : 0), box_ch = lane % chunks;
        const bool on = lane < (is_k ? 4 : 8) * chunks;
        const uint32_t ring = sbase + (is_k ? C::kOffK : C::kOffTmaV);
        const int bytes = is_k ? C::kKBytes : C::kTmaVBytes, slots = is_k ? C::kKSlots : C::kTmaVSlots;
        const uint32_t box = ring + (is_k ? box_ch * (64 * 128) + lane / chunks * 2048 : box_ch * (128 * 128) + box_page * 2048);
        const int el = is_k ? box_ch * kEl : (rank * (kDim / 2) + box_ch) * kEl;
        const int full = is_k ? kBarKFull : kBarVLanded, empty = is_k ? kBarKEmpty : kFp8 ? kBarRawEmpty : kBarVEmpty;
        const bool scl = kScl && is_k && lane >= 24;  // lanes that bring the tile's page scales
        const int page_of = scl ? lane - 24 : box_page;
        int tiles = 0;
        while (const volatile Piece* pc = take()) {
          const Span x{pc->x.klo, pc->x.khi, pc->x.nf, pc->x.w0, 0};
          const int n = pc->n, i0 = pc->i0, h = pc->h;
          const int* bt = p.block_table + (int64_t)pc->b * p.bt_s0;
          give_back();
          auto page_id = [&](int i) {
            const int page = tile_of(x, i0 + i) * (kKeys / kPageSize) + page_of;
            const uint32_t key = (uint32_t)page * kPageSize;
            const bool seen = i < n && (on || scl) && key < (uint32_t)x.khi &&
                              (key + kPageSize > (uint32_t)x.klo || key < (uint32_t)p.first_tokens);
            return seen ? bt[(int64_t)page * p.bt_s1] : -1;
          };
          float ks = 1.f, vs = 1.f;
          auto scales_of = [&](int id) {
            ks = vs = 1.f;
            if (scl && (unsigned)id < (unsigned)p.num_blocks) {
              ks = __ldg(p.k_scales + (int64_t)id * p.ks_s0 + (int64_t)h * p.ks_s1);
              vs = __ldg(p.v_scales + (int64_t)id * p.vs_s0 + (int64_t)h * p.vs_s1);
            }
          };
          int id = page_id(0), id1 = page_id(1);
          if (kScl) scales_of(id);
          for (int i = 0; i < n && ok; ++i) {
            const int cur = tiles + i, slot = cur % slots;
            if (cur >= slots && !wait_for(empty + slot, cur / slots - 1, 1)) break;
            if (kScl && is_k) {
              if (scl) {
                const float k1 = fminf(fmaxf(ks, kMinPageScale), kMaxPageScale);
                const float v1 = fminf(fmaxf(vs, kMinPageScale), kMaxPageScale);
                page_scale[cur % kScaleTiles * 8 + lane - 24] = make_float2(k1, log2f(v1));
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(kBarScales + cur % kScaleTiles));
              scales_of(id1);
            }
            if (lane == 0) {
              issued[is_k ? 0 : 1] = cur + 1;
              mbar_arrive_expect_tx(bar(full + slot), bytes);
            }
            __syncwarp();
            if (on)
              tma_load_4d(box + slot * bytes, is_k ? &tm_k : &tm_v, el, h, 0,
                          (unsigned)id < (unsigned)p.num_blocks ? id : p.num_blocks, bar(full + slot));
            __syncwarp();
            id = id1;
            id1 = page_id(i + 2);
          }
          tiles += n;
        }
      } else if (warp == kWarpMma) {
        // ======================= MMA issuer (the even CTA) ===============================
        // Q K^T of tile i + 1, then P V of tile i. The odd CTA's warp tells it that its half
        // of a K tile has landed.
        int tiles = 0, piece = 0;
        while (const volatile Piece* pc = take()) {
          const int n = pc->n;
          give_back();
          if (n == 0) continue;
          if (rank == 1) {
            for (int i = 0; i < n; ++i) {
              const int slot = (tiles + i) % C::kKSlots;
              if (!wait_for(kBarKFull + slot, (tiles + i) / C::kKSlots, 4)) break;
              if (lane == 0) mbar_arrive_cluster(lead(kBarKPeer + slot));
            }
            tiles += n;
            continue;
          }
          if (!wait_for(kBarQFull, piece, 2)) break;
          for (int i = 0; i <= n && ok; ++i) {
            if (i < n) {
              const int cur = tiles + i, slot = cur % C::kKSlots, use = cur / C::kKSlots;
              if (!wait_for(kBarKFull + slot, use, 4) || !wait_for(kBarKPeer + slot, use, 4)) break;
              tc_fence_after();
              const uint32_t src = sbase + C::kOffK + slot * C::kKBytes;
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  // bf16: 16 columns of d; e4m3: 32, of Q's first term, then of its second
                  const uint32_t ko = (uint32_t)((k & 3) * 32);
                  const uint64_t a = smem_desc(sbase + C::kOffQ + (k >> 2) * (128 * 128) + ko, 16, 1024, kLayoutSw128);
                  const uint64_t b = smem_desc(src + (kFp8 ? (k >> 2) & 1 : k >> 2) * (64 * 128) + ko, 16, 1024, kLayoutSw128);
                  if constexpr (kFp8)
                    mma_f8f6f4_pair(tmem + kColS + (cur & 1) * kKeys, a, b, C::kIdQK, k ? 1u : 0u);
                  else
                    mma_f16_pair(tmem + kColS + (cur & 1) * kKeys, a, b, C::kIdQK, k ? 1u : 0u);
                }
                mma_commit_pair(bar(kBarSFull + (cur & 1)));
                mma_commit_pair(bar(kBarKEmpty + slot));
                if (i == n - 1) mma_commit_pair(bar(kBarQFree));
              }
              __syncwarp();
            }
            if (i > 0) {
              const int cur = tiles + i - 1, slot = cur % C::kVSlots;
              if (!wait_for(kBarVFull + slot, cur / C::kVSlots, 4)) break;
              if (!wait_for(kBarPFull + (cur & 1), cur >> 1, 8)) break;
              if (i == 1 && piece > 0 && !wait_for(kBarOFree, piece - 1, 16)) break;
              tc_fence_after();
              const uint32_t src = sbase + C::kOffV + slot * C::kVBytes;
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  mma_f16_pair_ta(tmem + kColO, tmem + kColS + (cur & 1) * kKeys + 64 * (k >> 2) + 8 * (k & 3),
                                  smem_desc(src + k * 2048, 128 * 128, 1024, kLayoutSw128), C::kIdPV, i > 1 || k ? 1u : 0u);
                mma_commit_pair(bar(kBarPvDone + (cur & 1)));
                mma_commit_pair(bar(kBarVEmpty + slot));
              }
              __syncwarp();
            }
          }
          tiles += n;
          ++piece;
        }
        // every MMA has finished before the pair frees its memory
        if (rank == 0 && elect_one()) {
          mma_commit_pair(bar(kBarDrain));
          mbar_wait_drain(bar(kBarDrain), 0, kDrainLimitNs);
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (t0 < t1 && tid == 0) {
    // copies in flight land before the CTA ends, also when a role gave up; and the odd
    // CTA's copy of the last commit, so that no arrival is under way
    for (int k = issued[0] > C::kKSlots ? issued[0] - C::kKSlots : 0; k < issued[0]; ++k)
      mbar_wait_drain(bar(kBarKFull + k % C::kKSlots), (uint32_t)(k / C::kKSlots) & 1u, kDrainLimitNs);
    for (int k = issued[1] > C::kTmaVSlots ? issued[1] - C::kTmaVSlots : 0; k < issued[1]; ++k)
      mbar_wait_drain(bar(kBarVLanded + k % C::kTmaVSlots), (uint32_t)(k / C::kTmaVSlots) & 1u, kDrainLimitNs);
    if (rank == 1) mbar_wait_drain(bar(kBarDrain), 0, kDrainLimitNs);
  }
  __syncwarp();
  // both CTAs are done with each other's barriers and tensor memory
  cluster_arrive();
  __syncwarp();
  cluster_wait();
  if (warp == kWarpMma) tmem_dealloc_pair(tmem, kTmemCols);
}

// ---- the merge -------------------------------------------------------------------------
//
// CTA x takes the item that the share of pair x + 1 starts in, if it starts inside it
// and pair x holds the item's first tile: sums the pairs' partials in their order.
constexpr int kMergeThreads = 256, kMergeRows = 32;  // rows of a CTA, four at a time
constexpr int kMaxPairs = 256;

__global__ void __launch_bounds__(kMergeThreads) va_chunk_merge_kernel(const ChunkParams p) {
  __shared__ int s_slots[kMaxPairs];
  __shared__ int s_n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int c = blockIdx.x + 1;
  const int used = p.ws_start[0].used;
  if (c >= used) return;
  const ChunkStart st = p.ws_start[c];
  const Seq s = chunk_seq(p, st.b);
  const int row0 = st.m * kChunkRows + blockIdx.y * kMergeRows, rows = s.L * p.group;
  if (row0 >= rows) return;
  if (threadIdx.x < 32) {
    // the slots of the item's parts, in the pairs' order
    const int lane = threadIdx.x;
    const int64_t share = share_units(st.total, used);
    int n = 0;
    if (st.off < share_begin(st.total, share, c) && share_begin(st.total, share, c - 1) <= st.off) {
      const int tiles = item_span(p, s, st.m).n;
      for (int k0 = c - 1; k0 < used; k0 += 32) {
        const int k = k0 + lane;
        int64_t i0 = 0, i1 = 0;
        if (k < used) {
          i0 = ceil_units(p, share_begin(st.total, share, k) - st.off);
          i1 = ceil_units(p, share_begin(st.total, share, k + 1) - st.off);
          i1 = i1 < tiles ? i1 : tiles;
        }
        const unsigned has = __ballot_sync(0xffffffffu, i0 < i1);
        if (i0 < i1) s_slots[n + __popc(has & ((1u << lane) - 1))] = 2 * k + (i0 == 0 ? 1 : 0);
        n += __popc(has);
        if (has == 0) break;
      }
    }
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  if (n < 2) return;  // no item is split here, or an earlier pair's CTA joins it
  const float vd = p.v_descale ? *p.v_descale : 1.f;
  const int col = threadIdx.x % (kHeadDim / 4);
#pragma unroll 2
  for (int i = threadIdx.x / (kHeadDim / 4); i < kMergeRows; i += kMergeThreads / (kHeadDim / 4)) {
    const int row = row0 + i, r = blockIdx.y * kMergeRows + i;
    if (row >= rows) break;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < n; k0 += 4) {
      float2 ml[4];
      float4 a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < n) {
          const int64_t at = (int64_t)s_slots[k0 + k] * kChunkRows + r;
          ml[k] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml + at * 2));
          a[k] = __ldcg(reinterpret_cast<const float4*>(p.ws_acc + at * kHeadDim) + col);
        }
      }
      const float mc = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
      if (mc == -INFINITY) continue;
      const float w = M == -INFINITY ? 0.f : exp2f(M - mc);
      den *= w;
      acc.x *= w;
      acc.y *= w;
      acc.z *= w;
      acc.w *= w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (ml[k].x == -INFINITY) continue;  // no visible key: its partial holds nothing
        const float u = exp2f(ml[k].x - mc);
        den = fmaf(ml[k].y, u, den);
        acc.x = fmaf(a[k].x, u, acc.x);
        acc.y = fmaf(a[k].y, u, acc.y);
        acc.z = fmaf(a[k].z, u, acc.z);
        acc.w = fmaf(a[k].w, u, acc.w);
      }
      M = mc;
    }
    const int t = by_group(p, row), g = row - t * p.group;
    if (p.sinks && M != -INFINITY) den += exp2f(p.sinks[st.h * p.group + g] * kLog2e - M);
    const float inv = M != -INFINITY ? vd / den : 0.f;
    uint16_t* dst = p.out + (int64_t)(s.q0 + t) * p.o_s0 + (int64_t)(st.h * p.group + g) * p.o_s1 + 4 * col;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_b16x2(acc.x * inv, acc.y * inv), pack_b16x2(acc.z * inv, acc.w * inv));
  }
}

template <int KIND, bool VAR>
cudaError_t prepare_one(int32_t* max_pairs) {
  cudaError_t e = cudaFuncSetAttribute(va_chunk_kernel<KIND, VAR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<KIND>::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(Cfg<KIND>::kThreads);
  cfg.dynamicSmemBytes = Cfg<KIND>::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  e = cudaOccupancyMaxActiveClusters(&n, va_chunk_kernel<KIND, VAR>, &cfg);
  if (n < *max_pairs) *max_pairs = n;
  if (*max_pairs > kMaxPairs) *max_pairs = kMaxPairs;
  return e;
}

}  // namespace

cudaError_t prepare_chunk(int32_t* max_pairs) {
  *max_pairs = 1 << 20;
  cudaError_t e = prepare_one<kBf16, false>(max_pairs);
  if (e == cudaSuccess) e = prepare_one<kBf16, true>(max_pairs);
  if (e == cudaSuccess) e = prepare_one<kE4m3, false>(max_pairs);
  if (e == cudaSuccess) e = prepare_one<kE4m3, true>(max_pairs);
  if (e == cudaSuccess) e = prepare_one<kPageScaled, false>(max_pairs);
  if (e == cudaSuccess) e = prepare_one<kPageScaled, true>(max_pairs);
  return e;
}

template <int KIND>
static cudaError_t launch_main(cudaLaunchConfig_t& cfg, const ChunkParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v) {
  cfg.blockDim = dim3(Cfg<KIND>::kThreads);
  cfg.dynamicSmemBytes = Cfg<KIND>::kSmemBytes;
  return p.window_left >= 0 || p.softcap_log2 > 0.f ? cudaLaunchKernelEx(&cfg, va_chunk_kernel<KIND, true>, p, tm_k, tm_v)
                                                    : cudaLaunchKernelEx(&cfg, va_chunk_kernel<KIND, false>, p, tm_k, tm_v);
}

cudaError_t launch_chunk(const ChunkParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_v, cudaStream_t stream) {
  // programmatic dependents of the stream's previous kernel, as the verify kernels
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3(2 * p.pairs);
  const cudaError_t e = p.k_scales ? launch_main<kPageScaled>(cfg, p, tm_k, tm_v)
                        : p.kv_fp8 ? launch_main<kE4m3>(cfg, p, tm_k, tm_v)
                                   : launch_main<kBf16>(cfg, p, tm_k, tm_v);
  if (e != cudaSuccess || p.pairs < 2) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.pairs - 1, kChunkRows / kMergeRows);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, va_chunk_merge_kernel, p);
}

}  // namespace va
