// Split-KV main kernel over an absorbed-MLA latent cache (tcgen05, sm_103a).
//
// The grouped-head shared-KV verify kernel of sglang PR 34517 digest
// ("Implementation breakdown" item 1, the verify_mla.py excerpt) serves an
// absorbed-MLA layout: one KV head whose cache rows are [latent c (512) |
// rope key r (64)], logits (q_nope . c + q_pe . r) * sm_scale * k_scale, and
// the latent c as the value. All Hq heads x L draft tokens (<= 64 rows) of a
// sequence share every cache row, so each row is read from HBM once.
//
// The work split, the per-row online softmax in log2 units, the e4m3 hi/lo
// split of Q and, with block scales, of P and the bounded waits are those of the
// GQA kernel (va_main_tc.cu). What differs is the tensor-memory plan, which a
// 512-wide value forces. With Q and P split into two e4m3 terms stacked in the
// MMA's M (hi rows and lo rows), O would need 128 lanes x 512 fp32 columns, all
// of TMEM. So:
//  * S = Q K^T as before: M = 128 stacked rows (hi and lo of packed row
//    16q + i in lanes 32q + i and 32q + 16 + i), N = 64 keys, K = 576. The
//    latent part of Q is the A operand in TMEM (112 columns), its last 64
//    columns and the rope part a no-swizzle A operand in smem (16 KB); K is the
//    cache tile.
//  * O is kept transposed, O^T = V^T P^T: M = 128 latent columns per chunk,
//    N = the packed rows in use (a multiple of 16), K = keys. V^T is the cache
//    tile's latent part read as an MN-major A operand; P^T is a K-major B operand
//    in smem. Above 32 rows the two e4m3 terms of P are two MMAs into the same
//    accumulator (stacked in K), each with the block scales of its term; up to 32
//    rows a page-scaled call stacks them in N. O^T takes 4 chunks x 64 columns =
//    256 TMEM columns.
//  TMEM: O^T 0-255, two 64-column S tiles 256-383, Q latent 384-495, block
//  scales 496-511 (V's, all 1; P's, one set per P buffer).
// A cache tile is 64 keys = 4 pages; a page is 5 TMA boxes of 16 rows: four
// 128-byte latent chunks (128-byte swizzle) and the 64-byte rope part (64-byte
// swizzle, its own tensor map), so a tile fills four 8 KB regions and one of
// 4 KB; five ring slots (180 KB) are in flight, beside three P^T buffers (the
// tensor pipe runs Q K^T up to two tiles ahead of P V; four buffers, for which
// Q's second smem part leaves no room, would save 1 % of a 64-row call). A slot
// is freed after P V,
// since the same bytes are K and V. The cache loads carry an L2 evict_first
// policy, and the kernel is launched as a programmatic dependent of the
// stream's previous kernel (setup before griddepcontrol.wait), as in the GQA
// kernel.
// O^T columns are rows, so a rescale of some rows touches every lane: the
// softmax warps decide together, per tile, with one barrier reduction.
// FP8 cache only; plain attention (no window, soft cap or sinks).
#include "va_fp8.cuh"
#include "va_ptx.cuh"
#include "va_split.cuh"

namespace va {
namespace {

using namespace ptx;

constexpr int kT = kMlaTileKeys;               // 64 keys per tile
constexpr int kPagesPerTile = kT / kPageSize;  // 4
constexpr int kRegions = 5;                    // latent chunks 0-3, rope chunk 4
constexpr int kRegion = kT * 128;              // 8 KB: 64 rows x 128 bytes, 128-byte swizzle
constexpr int kPeRegion = kT * kMlaPe;         // 4 KB: 64 rows x 64 bytes, 64-byte swizzle
constexpr int kTileBytes = 4 * kRegion + kPeRegion;  // 36 KB
constexpr int kSlots = 5;
constexpr int kProducers = 3;                  // producer warps: each takes every third tile
// A producer's wait for a slot relies on its own previous wait (kProducers
// tiles back) to keep that slot's empty barrier within one phase.
static_assert(kProducers <= kSlots, "producers exceed the ring");
constexpr int kBoxes = kPagesPerTile * kRegions;  // 20 boxes per tile (16 of 2 KB, 4 of 1 KB)
constexpr uint32_t kPageBytes = 4 * 2048 + 1024;   // one page's boxes
static_assert(kBoxes <= 32, "one box per lane");
constexpr int kSBufs = 2;
constexpr int kPBufs = 3;                      // P^T buffers, and their block scales
constexpr int kPHalf = 64 * kT;                // one e4m3 term of P: 64 rows x 64 keys
constexpr int kPBuf = 2 * kPHalf;              // hi then lo
constexpr int kQkSteps = kMlaNope / 32;        // 16 K-steps over the latent part
constexpr int kQkTmemSteps = kQkSteps - 2;     // all but the last two from the TMEM A operand
constexpr int kQkPeSteps = kMlaPe / 32;        // 2 over the rope part
// the smem A operand: 128 stacked rows of the rope part and the last latent steps
constexpr int kQpeRow = kMlaPe + 32 * (kQkSteps - kQkTmemSteps);
constexpr int kQpeBytes = 128 * kQpeRow;
constexpr int kPvSteps = kT / 32;              // 2 K-steps of 32 keys
constexpr int kChunks = kMlaNope / 128;        // 4 O^T chunks of 128 latent columns

constexpr int kOffQpe = kSlots * kTileBytes;
constexpr int kOffP = kOffQpe + kQpeBytes;
constexpr int kOffX = kOffP + kPBufs * kPBuf;  // [2 parity][2 kh][64 rows] floats
constexpr int kOffSf = kOffX + 1024;           // per P buffer its block scales: [32 rows][4 row groups][4] bytes
constexpr int kOffBar = kOffSf + 512 * kPBufs;
constexpr int kOffSeqs = kOffBar + 2048;  // the batch's lengths (SeqMeta, kSeqCache)
constexpr int kSmemBytes = kOffSeqs + 16 * kSeqCache;
static_assert(kSmemBytes + 1024 <= 232448, "shared memory (with the 1 KB alignment slack)");
static_assert(kTileBytes % 1024 == 0 && kOffQpe % 1024 == 0, "swizzle atoms");

constexpr int kNarRows = 32;  // NAR: packed rows at most
__host__ __device__ constexpr int nar_p_buf(int rows) { return 2 * rows * kT; }  // both terms of P
// NAR in clusters, at most 16 rows: the latent part of Q on its way to tensor memory, in
// the P buffers' unused part: 16 rows of hi bytes, then of lo, a row's 16-byte
// groups g at g ^ (row % 8)
constexpr int kOffQStage = kOffP + kPBufs * nar_p_buf(16);
static_assert(kOffQStage + 2 * 16 * kMlaNope <= kOffX, "the staged Q fits behind the P buffers");
static_assert(nar_p_buf(kNarRows) <= kPBuf, "P buffers");

constexpr int kThreads = 512;  // 16 warps
constexpr int kSoftmaxThreads = 256;
constexpr int kBarAllSoftmax = 5;  // named barriers: 1-4 per quadrant, 5 all softmax warps

constexpr uint32_t kColO = 0;
constexpr uint32_t kColS = 256;
constexpr uint32_t kColQ = 384;
constexpr uint32_t kColSf = 496;  // block scales: V's (four columns, all 1), then P's (four per buffer)
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleOnes = 0x7F7F7F7Fu;
static_assert(kColQ + 8 * kQkTmemSteps <= kColSf && kColSf + 4 + 4 * kPBufs <= kTmemCols, "tensor memory");

constexpr uint32_t kIdQK = instr_desc(0, 0, false, kT, 128);         // e4m3 x e4m3, N = 64 keys
// A = V^T MN-major, N = the packed rows in use (a multiple of 16)
__device__ __forceinline__ uint32_t id_pv(int n) { return instr_desc_mx(false, n, 128, true); }

// A row's reference moves only when a tile's max passes m_ref + kFar, as in the
// GQA kernel; a move costs a CTA-wide pass over O^T.
constexpr float kFar = 32.f;

enum : int {
  kBarFull = 0,
  kBarEmpty = kBarFull + kSlots,
  kBarSFull = kBarEmpty + kSlots,
  kBarSFree = kBarSFull + kSBufs,
  kBarPFull = kBarSFree + kSBufs,
  kBarPFree = kBarPFull + kPBufs,
  kBarQFull = kBarPFree + kPBufs,
  kBarQFree,
  kBarOFull,
  kBarOFree,
  kBarDrain,
  kBarScales,  // page-scaled caches: a ring slot's page scales are written
  kNumBars = kBarScales + kSlots
};
// barrier area: mbarriers | TMEM address, abort flag | scan scratch (34 x 8) |
// last tile issued into each ring slot | per-row factors [2 rounds][64] floats
// at +1024 (2 KB in all); then the batch's lengths (1 KB)
constexpr int kOffTmemSlot = 8 * kNumBars;
constexpr int kOffScratch = 320;
constexpr int kOffSlotTile = kOffScratch + 34 * 8;  // last tile issued into each slot
constexpr int kOffRowVals = 1024;
constexpr int kOffScales = 1536;  // page-scaled: per ring slot its four pages' (scale, log2 of it)
static_assert(kOffScales + kSlots * kPagesPerTile * 8 <= 2048, "page scales");
static_assert(kOffTmemSlot + 8 <= kOffScratch && kOffSlotTile + 4 * kSlots <= kOffRowVals, "barrier area");

// Four bf16 values (two words) times 2^e -> e4m3 hi and lo bytes, in order.
__device__ __forceinline__ void split_q4(uint32_t wa, uint32_t wb, float up, uint32_t& hi, uint32_t& lo) {
  const float x0 = __uint_as_float(wa << 16) * up, x1 = __uint_as_float(wa & 0xFFFF0000u) * up;
  const float x2 = __uint_as_float(wb << 16) * up, x3 = __uint_as_float(wb & 0xFFFF0000u) * up;
  const uint32_t h01 = pack_fp8x2(x0, x1), h23 = pack_fp8x2(x2, x3);
  const float2 f01 = unpack_fp8x2(h01), f23 = unpack_fp8x2(h23);
  hi = h01 | (h23 << 16);
  lo = pack_fp8x2(x0 - f01.x, x1 - f01.y) | (pack_fp8x2(x2 - f23.x, x3 - f23.y) << 16);
}

__device__ __forceinline__ float bf16_amax2(uint32_t w) {
  return fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xFFFF0000u)));
}

// The power of two that takes a row of largest |value| amax into [2^7, 2^8).
__device__ __forceinline__ int q_exponent(float amax) {
  if (!(amax > 0.f && amax < INFINITY)) return 0;
  const int e = 7 - ((int)((__float_as_uint(amax) >> 23) & 0xFF) - 127);
  return e < -120 ? -120 : (e > 120 ? 120 : e);
}

// Byte offset of element (row m, column k) in a no-swizzle K-major operand
// whose rows are `row_bytes` long: 8-row x 16-byte core matrices, K-adjacent
// ones 128 bytes apart, 8-row groups 8 * row_bytes apart.
__device__ __forceinline__ int core_off(int m, int k, int row_bytes) {
  return (m >> 3) * (8 * row_bytes) + (k >> 4) * 128 + (m & 7) * 16 + (k & 15);
}

// SCL: a page-scaled cache, one scale a page for keys and values; as in the
// GQA kernel it multiplies the page's logits, and as the value's scale joins
// the weight, P = 2^(s + log2 scale - e), with l summing P / scale. A
// thread's 16 keys of a tile are one page. The producers bring the scales
// with the ring slot. 64 sequences of 8K to 32K keys (733 MB), 16 heads: 153 us
// with 3 draft tokens, 135 with one, 71 and 82 % of the measured copy bandwidth;
// of the 153 the merge kernel is 11.
// CLU: one cluster of CTAs per item, as in the GQA kernel: two sequences of
// 1,024 and 769 keys 10.4 to 10.9 us a call (22.1 split over all CTAs).
// NAR: at most 32 packed rows. P's two terms are then stacked in the N of P V
// (rows r and nar + r of P^T, columns r and nar + r of O^T, added up in the
// epilogue): half its instructions, and N = 32 for 16 rows (64 sequences of 8K
// to 32K, one token: N = 64 135.9 us, N = 32 132.5). P's exponents are packed fp32
// FMAs, two keys an instruction (137.8 -> 135.2; at 64 rows 201 -> 204).
template <bool SCL, bool CLU, bool NAR>
__global__ void __launch_bounds__(kThreads, 1)
    va_mla_tc_kernel(const Params p, const __grid_constant__ CUtensorMap tm_kv,
                     const __grid_constant__ CUtensorMap tm_pe) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kOffBar + kOffTmemSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kOffBar + kOffTmemSlot + 4);
  long long* scratch = reinterpret_cast<long long*>(sm + kOffBar + kOffScratch);  // 32 slots
  long long* s_ts = scratch + 32;
  int* s_j = reinterpret_cast<int*>(scratch + 33);
  float* xch = reinterpret_cast<float*>(sm + kOffX);
  float* row_vals = reinterpret_cast<float*>(sm + kOffBar + kOffRowVals);  // [2][64]
  volatile int* slot_tile = reinterpret_cast<volatile int*>(sm + kOffBar + kOffSlotTile);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int c = blockIdx.x;
  const uint32_t sbase = smem_addr(sm);
  auto bar = [&](int i) { return smem_addr(&bars[i]); };

  // The merge kernel is a programmatic dependent; it waits for this grid.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- setup (no global memory: runs while the stream's previous kernel ends) ---
  constexpr uint32_t kSwWarps = kSoftmaxThreads / 32;
  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar(kBarFull + s), 1);
      mbar_init(bar(kBarEmpty + s), 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarSFree + i), kSwWarps);
    }
    for (int i = 0; i < kPBufs; ++i) {
      mbar_init(bar(kBarPFull + i), kSwWarps);
      mbar_init(bar(kBarPFree + i), 1);
    }
    mbar_init(bar(kBarQFull), kSwWarps);
    mbar_init(bar(kBarQFree), 1);
    mbar_init(bar(kBarOFull), 1);
    mbar_init(bar(kBarOFree), kSwWarps);
    mbar_init(bar(kBarDrain), 2);
    if constexpr (SCL)
      for (int s = 0; s < kSlots; ++s) mbar_init(bar(kBarScales + s), 1);
    *abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) slot_tile[s] = -1;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0 && p.num_blocks > 0) {
    tma_prefetch_desc(&tm_kv);
    tma_prefetch_desc(&tm_pe);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A programmatic dependent of the stream's previous kernel (which may write
  // Q, the block table or the lengths, and may still read this workspace):
  // nothing global is read or written before its completion.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  long long t0, t1, ts_first = 0;
  int j_first = 0;
  bool seqs_cached = false;
  SeqMeta meta{};  // CLU: the item's lengths
  if constexpr (CLU) {
    meta = locate_cluster_work(p, c, p.cluster, &t0, &t1, &j_first, reinterpret_cast<SeqMeta*>(sm + kOffSeqs));
    seqs_cached = p.num_seqs <= kSeqCache;
  } else {
    locate_work<kThreads>(p, c, scratch, s_j, s_ts, &t0, &t1, &j_first, &ts_first,
                          reinterpret_cast<SeqMeta*>(sm + kOffSeqs), &seqs_cached);
  }
  const SeqMeta* seqs = seqs_cached ? reinterpret_cast<const SeqMeta*>(sm + kOffSeqs) : nullptr;
  if (!CLU && t0 >= t1) {  // CTA-uniform
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    return;
  }
  // CLU: the partial's rows in the drained ring, then (m, l)
  constexpr int kOffMl = kMaxRows * kMlaNope * 4;
  static_assert(!CLU || kOffMl + kMaxRows * 8 <= kOffQpe, "the partial fits in the ring");
  float* part = reinterpret_cast<float*>(sm);
  float* part_ml = reinterpret_cast<float*>(sm + kOffMl);
  if (warp >= 4 && warp < 12) {
    // the first item's Q rows into L2 before the ring's first loads flood HBM
    int jq = j_first;
    long long tq = ts_first;
    Piece pq;
    if (next_piece(p, t0, t1, jq, tq, pq, seqs)) {
      const int r = 16 * (warp & 3) + (lane & 15), qtr = 2 * ((warp - 4) >> 2) + (lane >> 4);
      if (r < pq.R) {
        const uint16_t* src =
            p.q + (int64_t)(pq.q0 + r / p.group) * p.q_s0 + (int64_t)(pq.kvh * p.group + r % p.group) * p.q_s1;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 128 * qtr));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 128 * qtr + 64));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + kMlaNope + 16 * qtr));
      }
    }
  }


  // With at most 48 packed rows the softmax warps of quadrant 3 are idle; the
  // two MMA issuers then sit on that quadrant's scheduler, where no ALU work
  // competes with them (latent mid context, 48 rows: 158.4 -> 156.7 us, 16
  // rows 134.3 -> 131.9).
  const int nar = p.max_rows <= 16 ? 16 : 32;  // NAR: P's low terms are rows nar ... of P^T
  const bool alt = p.max_rows <= 48;
  const int prod = alt ? (warp < 3 ? warp : -1) : (warp == 0 ? 0 : (warp == 2 || warp == 3) ? warp - 1 : -1);
  const bool qk_warp = warp == (alt ? 3 : 1), pv_warp = warp == (alt ? 15 : 12);
  if (CLU && t0 >= t1) {
    if (tid < kMaxRows) {
      part_ml[2 * tid] = -INFINITY;
      part_ml[2 * tid + 1] = 0.f;
    }
  } else if (prod >= 0) {
    // ======================= TMA producers ======================================
    const uint64_t kv_policy = l2_evict_first_policy();  // the cache rows are read once
    int it = 0;
    int j = j_first;
    long long ts = ts_first;
    Piece pc;
    bool ok = true;
    while (ok && next_piece(p, t0, t1, j, ts, pc, seqs)) {
      const int npages = (pc.S + kPageSize - 1) / kPageSize;
      const int* bt_row = p.block_table + (int64_t)pc.b * p.bt_s0;
      int win = -1;
      int my_page = -1;
      ScaleWindow sw;
      for (int lt = pc.lt0; lt < pc.lt1 && ok; ++lt, ++it) {
        if (it % kProducers != prod) continue;
        const int s = it % kSlots;
        const int pg0 = lt * kPagesPerTile;
        if constexpr (SCL) {
          // this warp's tiles of a window start 0, 12 and 24 pages into it
          if (win < 0 || pg0 + kPagesPerTile > win + 32) {
            win = pg0;
            sw.move(p, bt_row, 0, win, 36, 0, npages);
            my_page = sw.id;
          } else {
            sw.advance(p, 0);
          }
        } else if (win < 0 || pg0 + kPagesPerTile > win + 32) {
          win = pg0;
          const int pg = win + lane;
          my_page = pg < npages ? bt_row[(int64_t)pg * p.bt_s1] : -1;
          if (lane == 0 && win + 32 < npages)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(bt_row + (int64_t)(win + 32) * p.bt_s1));
        }
        uint32_t nvalid = 0;
        int ids[kPagesPerTile];
#pragma unroll
        for (int i = 0; i < kPagesPerTile; ++i) {
          ids[i] = __shfl_sync(0xffffffffu, my_page, pg0 + i - win);
          const bool v = (pg0 + i) < npages && (unsigned)ids[i] < (unsigned)p.num_blocks;
          ids[i] = v ? ids[i] : -1;
          nvalid += v ? 1u : 0u;
        }
        const bool got = __all_sync(
            0xffffffffu, mbar_wait(bar(kBarEmpty + s), ((it / kSlots) & 1) ^ 1, abort_flag, p.wait_limit_ns));
        if (!got) {
          if (lane == 0) fail(p, abort_flag, 1);
          ok = false;
          break;
        }
        const uint32_t dst = sbase + s * kTileBytes;
        if (lane == 0) {
          slot_tile[s] = it;
          mbar_arrive_expect_tx(bar(kBarFull + s), nvalid * kPageBytes);
        }
        __syncwarp();
        if (lane < kBoxes) {  // lane -> (page, 128-byte latent chunk or the 64-byte rope)
          const int i = lane / kRegions, ch = lane % kRegions;
          int id = ids[0];
#pragma unroll
          for (int u = 1; u < kPagesPerTile; ++u)
            if (i == u) id = ids[u];
          if (id >= 0) {
            if (ch < 4)
              tma_load_4d_hint(dst + ch * kRegion + i * 2048, &tm_kv, ch * 128, 0, 0, id, bar(kBarFull + s),
                               kv_policy);
            else
              tma_load_4d_hint(dst + 4 * kRegion + i * 1024, &tm_pe, kMlaNope, 0, 0, id, bar(kBarFull + s),
                               kv_policy);
          }
        }
        if constexpr (SCL) {
          const int i = win + lane - pg0;
          if (i >= 0 && i < kPagesPerTile)
            reinterpret_cast<float2*>(sm + kOffBar + kOffScales)[s * kPagesPerTile + i] =
                softmax_scales(sw.ks, sw.vs);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarScales + s));
        }
        __syncwarp();
      }
    }
    // Copies still in flight land before the CTA goes away, also when another
    // role gave up (the window: see the GQA kernel's producers).
    if (lane == 0) {
      for (int k = (it > kSlots + kProducers - 1 ? it - kSlots - kProducers + 1 : 0); k < it; ++k) {
        if (k % kProducers != prod) continue;
        drain_ring_tile(bar(kBarFull + k % kSlots), k, kSlots, slot_tile + k % kSlots, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else if (qk_warp || pv_warp) {
    // ======================= MMA issuers ==========================================
    const bool is_qk = qk_warp;
    const uint32_t qpe = sbase + kOffQpe;
    const uint32_t idpv = id_pv(NAR ? 2 * nar : (p.max_rows + 15) & ~15);
    int it = 0, piece_idx = 0;
    int j = j_first;
    long long ts = ts_first;
    Piece pc;
    bool ok = true;
    // The whole warp walks the tiles and waits, with one vote a tile, and one
    // elected thread issues. In a branch that only one lane enters, every
    // operand of every tcgen05.mma is a lane's value that has to be moved to
    // the warp's registers first, and an MMA of N = 64 costs its issuer about
    // 50 cycles; so the issue, and not the tensor cores, was the bound (latent
    // mid context, page-scaled, 48 rows 175.4 -> 159.1 us, 16 rows 162.2 ->
    // 135; with one descale 180.1 -> 157.4).
    auto arrived = [&](int b, uint32_t par) { return mbar_wait(bar(b), par, abort_flag, p.wait_limit_ns); };
    auto all_or_fail = [&](bool got, int code) {
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) fail(p, abort_flag, code);
        ok = false;
      }
      return ok;
    };
    while (ok && next_piece(p, t0, t1, j, ts, pc, seqs)) {
      const int first = __shfl_sync(0xffffffffu, it, 0);
      const int ntile = __shfl_sync(0xffffffffu, pc.lt1 - pc.lt0, 0);
      if (is_qk) {
        if (!all_or_fail(arrived(kBarQFull, piece_idx & 1), 2)) break;
        tc_fence_after();
        for (int i = 0; i < ntile && ok; ++i) {
          const int cur = first + i;
          const int s = cur % kSlots;
          const int b = cur & (kSBufs - 1);
          bool got = arrived(kBarFull + s, (cur / kSlots) & 1);
          if (cur >= kSBufs) got = got && arrived(kBarSFree + b, ((cur - kSBufs) / kSBufs) & 1);
          if (!all_or_fail(got, 32)) break;
          tc_fence_after();
          const uint32_t kst = sbase + s * kTileBytes;
          const uint32_t d = tmem + kColS + b * kT;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kQkSteps; ++k) {
              const uint64_t bdesc = smem_desc(kst + (k >> 2) * kRegion + (k & 3) * 32, 16, 1024, kLayoutSw128);
              if (k < kQkTmemSteps)
                mma_f8f6f4_ta(d, tmem + kColQ + 8 * k, bdesc, kIdQK, k ? 1u : 0u);
              else
                mma_f8f6f4(d, smem_desc(qpe + (kQkPeSteps + k - kQkTmemSteps) * 256, 128, 8 * kQpeRow, kLayoutNone), bdesc,
                           kIdQK, 1u);
            }
#pragma unroll
            for (int k = 0; k < kQkPeSteps; ++k) {
              const uint64_t adesc = smem_desc(qpe + k * 256, 128, 8 * kQpeRow, kLayoutNone);
              const uint64_t bdesc = smem_desc(kst + 4 * kRegion + k * 32, 16, 512, kLayoutSw64);
              mma_f8f6f4(d, adesc, bdesc, kIdQK, 1u);
            }
            mma_commit(bar(kBarSFull + b));
            if (i == ntile - 1) mma_commit(bar(kBarQFree));
          }
          __syncwarp();
        }
      } else {
        for (int i = 0; i < ntile && ok; ++i) {
          const int x = first + i;
          const int pb = x % kPBufs;
          const int s = x % kSlots;
          bool got = arrived(kBarPFull + pb, (x / kPBufs) & 1) && arrived(kBarFull + s, (x / kSlots) & 1);
          if (i == 0 && piece_idx > 0) got = got && arrived(kBarOFree, (piece_idx - 1) & 1);
          if (!all_or_fail(got, 4)) break;
          tc_fence_after();
          const uint32_t kst = sbase + s * kTileBytes;
          const uint32_t pbuf = sbase + kOffP + pb * (NAR ? nar_p_buf(nar) : kPBuf);
          if (elect_one()) {
            const uint32_t sf = tmem + kColSf + 4 + 4 * pb;
            tmem_cp_scales(sf, smem_desc(sbase + kOffSf + 512 * pb, 0, 128, kLayoutNone));
#pragma unroll
            for (int kk = 0; kk < kPvSteps; ++kk) {
              const uint64_t bhi = smem_desc(pbuf + kk * 256, 128, 8 * kT, kLayoutNone);
              const uint64_t blo = smem_desc(pbuf + kPHalf + kk * 256, 128, 8 * kT, kLayoutNone);
#pragma unroll
              for (int a = 0; a < kChunks; ++a) {
                // V^T chunk a: latent columns [128 a, +128) of keys [32 kk, +32)
                const uint64_t adesc = smem_desc(kst + a * kRegion + kk * 4096, kRegion, 1024, kLayoutSw128);
                const uint32_t d = tmem + kColO + 64 * a;
                mma_mxf8(d, adesc, bhi, idpv | ((uint32_t)kk << 4), tmem + kColSf, sf,
                         (i == 0 && kk == 0) ? 0u : 1u);
                if constexpr (!NAR)
                  mma_mxf8(d, adesc, blo, idpv | ((uint32_t)(kPvSteps + kk) << 4), tmem + kColSf, sf, 1u);
              }
            }
            mma_commit(bar(kBarPFree + pb));
            mma_commit(bar(kBarEmpty + s));
            if (i == ntile - 1) mma_commit(bar(kBarOFull));
          }
          __syncwarp();
        }
      }
      it = first + ntile;
      ++piece_idx;
    }
    if (elect_one()) {
      mma_commit(bar(kBarDrain));
      mbar_wait_drain(bar(kBarDrain), 0, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ======================= softmax / epilogue ===================================
    const int q = warp & 3;              // TMEM lane quadrant
    const int kh = (warp - 4) >> 2;      // half of each tile's keys, half of the O^T chunks
    const int sub = lane >> 4;
    const int rl = lane & 15;
    const int r = 16 * q + rl;           // packed row
    const int qtr = 2 * kh + sub;        // key quarter (16 keys) of a tile
    const uint32_t lane_base = (uint32_t)(32 * q) << 16;
    const float kd = p.k_descale ? *p.k_descale : 1.0f;
    // The logit scale is kept positive (the softmax takes the max of the raw
    // dot products and applies the scale after): a negative scale negates Q
    // as it is staged, and a zero one becomes a tiny positive one.
    const float cscale_signed = p.scale_log2 * kd;
    const float cscale = fmaxf(fabsf(cscale_signed), 1e-30f);
    const bool q_neg = cscale_signed < 0.f;
    const int G = p.group;
    unsigned char* qpe_s = sm + kOffQpe;
    int it = 0, piece_idx = 0, round = 0;
    int j = j_first;
    long long ts = ts_first;
    Piece pc;
    bool ok = true;
    // Waits are warp-uniform; after a failure the warp walks the same pieces
    // and tiles "dry" so that every named barrier still sees all its threads.
    auto wait_or_fail = [&](int b, uint32_t par, int code) {
      if (!ok) return false;
      const bool got = __all_sync(0xffffffffu, mbar_wait(bar(b), par, abort_flag, p.wait_limit_ns));
      if (!got) {
        if (lane == 0) fail(p, abort_flag, code);
        ok = false;
      }
      return ok;
    };
    // S of tile cur, page-scaled its pages' scales, and the P buffer that P V of
    // tile cur - kPBufs read, with one vote
    auto wait_tile = [&](int cur) {
      if (!ok) return false;
      bool got = true;
      if constexpr (SCL)
        got = mbar_wait(bar(kBarScales + cur % kSlots), (cur / kSlots) & 1, abort_flag, p.wait_limit_ns);
      got = got && mbar_wait(bar(kBarSFull + (cur & (kSBufs - 1))), (cur / kSBufs) & 1, abort_flag, p.wait_limit_ns);
      if (cur >= kPBufs)
        got = got && mbar_wait(bar(kBarPFree + cur % kPBufs), ((cur - kPBufs) / kPBufs) & 1, abort_flag, p.wait_limit_ns);
      got = __all_sync(0xffffffffu, got);
      if (!got) {
        if (lane == 0) fail(p, abort_flag, 256);
        ok = false;
      }
      return ok;
    };
    // Row-wide combine over the row's four threads (lanes t, t ^ 16 of this
    // warp and of the quadrant's other warp), as in the GQA kernel.
    int xround = 0;
    auto exchange = [&](float v, bool is_max) {
      v = is_max ? fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16)) : v + __shfl_xor_sync(0xffffffffu, v, 16);
      const int par = xround & 1;
      ++xround;
      if (sub == 0) xch[(par * 2 + kh) * 64 + r] = v;
      named_bar(1 + q, 64);
      const float other = xch[(par * 2 + (kh ^ 1)) * 64 + r];
      return is_max ? fmaxf(v, other) : v + other;
    };
    // This lane's last 16 words of Q's latent part (columns 448 on) go to the smem
    // A operand, behind the rope part: their place in tensor memory holds the block
    // scales.
    auto store_tail = [&](const uint32_t (&d)[16]) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(qpe_s + core_off(32 * q + lane, kMlaPe + 16 * i, kQpeRow)) =
            make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]);
    };
    // V's block scales are 1 (P's, in the columns behind, come with every tile)
    if (kh == 0) {
      tmem_fill_32x32b_x8(tmem + lane_base + kColSf, kScaleOnes);
      tmem_wait_st();
    }
    // Q of piece pq: latent columns [128 qtr, +128) and rope columns
    // [16 qtr, +16) of row r, scaled by 2^e and split into e4m3 hi and lo.
    // The latent part goes to the TMEM A operand (hi row in lane 32q + rl, lo
    // row in lane 32q + 16 + rl, four columns a word), its last 64 columns and
    // the rope part to the smem A operand. Returns the row's logit scale.
    auto stage_q = [&](const Piece& pq, int qidx) -> float {
      if (qidx > 0) wait_or_fail(kBarQFree, (qidx - 1) & 1, 128);
      const bool row_ok = r < pq.R;
      const int tq = row_ok ? r / G : 0;
      const int gq = row_ok ? r - tq * G : 0;
      const uint16_t* src = p.q + (int64_t)(pq.q0 + tq) * p.q_s0 + (int64_t)(pq.kvh * G + gq) * p.q_s1;
      // the row's largest |value| first (over its four threads), then the
      // conversion, re-reading the 288 bytes (cache hits)
      const bool ld = ok && row_ok;
      const uint4* nsrc = reinterpret_cast<const uint4*>(src + 128 * qtr);
      const uint4* psrc = reinterpret_cast<const uint4*>(src + kMlaNope + 16 * qtr);
      float amax = 0.f;
      if (ld) {
#pragma unroll
        for (int i = 0; i < 18; ++i) {
          const uint4 a = i < 16 ? nsrc[i] : psrc[i - 16];
          amax = fmaxf(amax, fmaxf(fmaxf(bf16_amax2(a.x), bf16_amax2(a.y)),
                                   fmaxf(bf16_amax2(a.z), bf16_amax2(a.w))));
        }
      }
      amax = exchange(amax, true);
      const int e = q_exponent(amax);
      const float up = __uint_as_float((uint32_t)(e + 127) << 23) * (q_neg ? -1.f : 1.f);
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      if (ok) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // own columns [128 qtr + 64 hf, +64): 16 words of hi and of lo
          uint32_t hw[16], lw[16];
#pragma unroll
          for (int w = 0; w < 16; w += 2) {
            const uint4 a = ld ? nsrc[8 * hf + (w >> 1)] : make_uint4(0, 0, 0, 0);
            split_q4(a.x, a.y, up, hw[w], lw[w]);
            split_q4(a.z, a.w, up, hw[w + 1], lw[w + 1]);
          }
          // sub 0 (hi lane) takes the hi terms of both threads' columns, sub 1
          // (lo lane) the lo terms: trade the part the partner's lane takes
          uint32_t d1[16], d2[16];
#pragma unroll
          for (int w = 0; w < 16; ++w) {
            const uint32_t recv = __shfl_xor_sync(0xffffffffu, sub ? hw[w] : lw[w], 16);
            d1[w] = sub ? recv : hw[w];   // columns of sub 0's span
            d2[w] = sub ? lw[w] : recv;   // columns of sub 1's span
          }
          tmem_st_32x32b_x16(tmem + lane_base + kColQ + 64 * kh + 16 * hf, d1);
          if (kh == 1 && hf == 1)
            store_tail(d2);
          else
            tmem_st_32x32b_x16(tmem + lane_base + kColQ + 64 * kh + 32 + 16 * hf, d2);
        }
        uint32_t ph[4], pl[4];
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
          const uint4 a = ld ? psrc[w >> 1] : make_uint4(0, 0, 0, 0);
          split_q4(a.x, a.y, up, ph[w], pl[w]);
          split_q4(a.z, a.w, up, ph[w + 1], pl[w + 1]);
        }
        const int mh = 32 * q + rl, ml = mh + 16;
        *reinterpret_cast<uint4*>(qpe_s + core_off(mh, 16 * qtr, kQpeRow)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        *reinterpret_cast<uint4*>(qpe_s + core_off(ml, 16 * qtr, kQpeRow)) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull));
      }
      return cscale * down;  // rows past R stage zeros: their logits are 0
    };
    // The same in a cluster whose rows are one quadrant's (there it is the start
    // that counts): the quadrant's two warps alone would convert 144 columns a
    // thread. Here sixteen threads share a row, each
    // with its loads in flight at once and the row's max by shuffles; the
    // converted latent part goes through shared memory to the quadrant's
    // warps, which move it to the TMEM operand; the rows' factors through
    // row_vals[48, 64), which no rescale of 16 rows uses (two sequences of 1,024 and 769
    // keys 11.9 -> 10.6 us; in the split over all CTAs its
    // registers cost the tile loop 1 to 4 %).
    auto stage_q16 = [&](const Piece& pq, int qidx) -> float {
      const int row = (tid - 128) >> 4, cc = tid & 15;
      const bool ld = ok && row < pq.R;
      uint4 x[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) x[i] = make_uint4(0, 0, 0, 0);
      if (ld) {
        const int tq = row / G, gq = row - tq * G;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(pq.q0 + tq) * p.q_s0 +
                                                          (int64_t)(pq.kvh * G + gq) * p.q_s1);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = src[16 * i + cc];
        if (cc < 8) x[4] = src[64 + cc];
      }
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 5; ++i)
        amax = fmaxf(amax, fmaxf(fmaxf(bf16_amax2(x[i].x), bf16_amax2(x[i].y)),
                                 fmaxf(bf16_amax2(x[i].z), bf16_amax2(x[i].w))));
#pragma unroll
      for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = q_exponent(amax);
      const float up = __uint_as_float((uint32_t)(e + 127) << 23) * (q_neg ? -1.f : 1.f);
      unsigned char* stage = sm + kOffQStage + row * kMlaNope;
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        split_q4(x[i].x, x[i].y, up, hi[0], lo[0]);
        split_q4(x[i].z, x[i].w, up, hi[1], lo[1]);
        const int c8 = 16 * i + cc;  // eight columns
        const int off = (((c8 >> 1) ^ (row & 7)) << 4) + ((c8 & 1) << 3);
        *reinterpret_cast<uint2*>(stage + off) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(stage + 16 * kMlaNope + off) = make_uint2(lo[0], lo[1]);
      }
      if (cc == 0) row_vals[48 + row] = __uint_as_float((uint32_t)(127 - e) << 23);
      if (qidx > 0) wait_or_fail(kBarQFree, (qidx - 1) & 1, 128);
      if (ok && cc < 8) {
        split_q4(x[4].x, x[4].y, up, hi[0], lo[0]);
        split_q4(x[4].z, x[4].w, up, hi[1], lo[1]);
        *reinterpret_cast<uint2*>(qpe_s + core_off(row, 8 * cc, kQpeRow)) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(qpe_s + core_off(16 + row, 8 * cc, kQpeRow)) = make_uint2(lo[0], lo[1]);
      }
      named_bar(kBarAllSoftmax, kSoftmaxThreads);
      const float down = row_vals[48 + rl];
      if (ok) {
        if (q == 0) {
          // this lane's TMEM row: hi of row rl, or lo; columns [256 kh, +256)
          const unsigned char* src = sm + kOffQStage + sub * (16 * kMlaNope) + rl * kMlaNope;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t d[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(src + (((16 * kh + 4 * h + i) ^ (rl & 7)) << 4));
              d[4 * i] = v.x;
              d[4 * i + 1] = v.y;
              d[4 * i + 2] = v.z;
              d[4 * i + 3] = v.w;
            }
            if (kh == 1 && h == 3)
              store_tail(d);
            else
              tmem_st_32x32b_x16(tmem + lane_base + kColQ + 64 * kh + 16 * h, d);
          }
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull));
      }
      return cscale * down;
    };
    auto stage = [&](const Piece& pq, int qidx) -> float {
      if constexpr (NAR && CLU)
        if (nar == 16) return stage_q16(pq, qidx);
      return stage_q(pq, qidx);
    };
    // The next piece's Q segments of this thread (three 128-byte lines) into
    // L2, a piece ahead: under full HBM load a round trip to DRAM takes
    // several microseconds, and staging Q sits on the softmax's path.
    auto prefetch_q = [&](const Piece& pq) {
      if (r < pq.R) {
        const int tq = r / G, gq = r - tq * G;
        const uint16_t* src = p.q + (int64_t)(pq.q0 + tq) * p.q_s0 + (int64_t)(pq.kvh * G + gq) * p.q_s1;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 128 * qtr));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 128 * qtr + 64));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + kMlaNope + 16 * qtr));
      }
    };
    float rs_next = 0.f;
    bool staged_next = false;
    while (next_piece(p, t0, t1, j, ts, pc, seqs)) {
      Piece pn;
      int jn = j;
      long long tsn = ts;
      const bool has_next = next_piece(p, t0, t1, jn, tsn, pn, seqs);
      const float rs = staged_next ? rs_next : stage(pc, piece_idx);
      staged_next = false;
      if (has_next) prefetch_q(pn);
      const bool row_ok = r < pc.R;
      const int tq = row_ok ? r / G : 0;

      // a quadrant none of whose 16 rows is in use has no S to read and no P to
      // write (its P rows reach only output columns that are never read); it
      // takes part in the votes, the rescales, the epilogue
      const bool idle = 16 * q >= pc.R;
      float m_ref = -INFINITY;
      float l = 0.f;
      const int vis_end = pc.S - pc.L + tq;  // last visible key of this row
      const int first = it;
      for (int lt = pc.lt0; lt < pc.lt1; ++lt, ++it) {
        const int cur = it;
        const int b = cur & (kSBufs - 1);
        const int pb = cur % kPBufs;
        if (lt == pc.lt1 - 1 && has_next) {
          rs_next = stage(pn, piece_idx + 1);
          staged_next = true;
        }
        float x[16];  // logits of keys [16 qtr, +16) of this tile, this row
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = -INFINITY;
        // the factor of the raw dot products (a positive normal number: -inf
        // stays -inf) and, page-scaled, the offset log2 scale of the page
        float xs = rs, lv = 0.f;
        const bool here = wait_tile(cur);
        if (SCL && here) {
          const float2 sc =
              reinterpret_cast<const float2*>(sm + kOffBar + kOffScales)[(cur % kSlots) * kPagesPerTile + qtr];
          xs = fmaxf(rs * sc.x, 1.2e-38f);
          lv = sc.y;
        }
        if (idle) {
          if (here && lane == 0) mbar_arrive(bar(kBarSFree + b));
        } else if (here) {
          tc_fence_after();
          // the hi and lo partials of row r, keys [32 kh + 16 sub, +16): two
          // 16-lane loads (hi rows in lanes 32q.., lo rows in lanes
          // 32q + 16..) whose second halves go to threads 16-31
          uint32_t vh[16], vl[16];
          tmem_ld_16x32bx2_x16<16>(tmem + lane_base + kColS + b * kT + 32 * kh, vh);
          tmem_ld_16x32bx2_x16<16>(tmem + lane_base + (16u << 16) + kColS + b * kT + 32 * kh, vl);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarSFree + b));
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(vh[i]) + __uint_as_float(vl[i]);
          const int key0 = lt * kT + 16 * qtr;
          if (lt * kT + kT - 1 > pc.S - pc.L) {  // tail tile: causal mask
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (key0 + i > vis_end) x[i] = -INFINITY;
          }
        }
        float top = -INFINITY;  // of this thread's raw dot products; xs > 0 keeps the order
#pragma unroll
        for (int i = 0; i < 16; i += 2) top = fmax3(top, x[i], x[i + 1]);
        const float tmax = SCL ? fmaf(top, xs, lv) : top * xs;
        const float bmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 16));  // of a block of P
        // A row's reference moves only when one of its four threads sees a key
        // above m_ref + kFar. One vote over all softmax threads finds out (an
        // item's first tile sets the references: no vote); only then is the row
        // max exchanged.
        float m_new = m_ref, alpha = 1.f;
        bool any = false;
        float* al = row_vals + (round & 1) * 64;
        ++round;
        if (cur == first || named_bar_or(kBarAllSoftmax, kSoftmaxThreads, ok && tmax > m_ref + kFar)) {
          const float rmax = exchange(tmax, true);
          const bool need = ok && rmax > m_ref + kFar;
          m_new = need ? floorf(rmax) : m_ref;
          if (cur != first) {
            const bool rescale = need && (m_ref != -INFINITY);
            alpha = rescale ? ex2(m_ref - m_new) : 1.f;
            // O^T keeps a row in a column across all 128 lanes: every softmax
            // warp scales its lanes' part of the rows that moved, so the
            // decision is taken by all of them at once
            if (kh == 0 && sub == 0 && (!NAR || r < nar)) {
              al[r] = alpha;
              if constexpr (NAR) al[nar + r] = alpha;
            }
            any = named_bar_or(kBarAllSoftmax, kSoftmaxThreads, rescale);
          }
        }
        if (!ok) continue;

        float ls = 0.f;
        if (!idle) {
          // P = 2^(s - e), e the block's exponent (va_fp8.cuh); 0 without a visible key
          uint32_t ph[4], pl[4];
          const float e = block_exponent(bmax, m_new);
          const float off2 = lv - e;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float a, bb;
            if constexpr (NAR) {
              unpack2(fma2(pack2(x[2 * i], x[2 * i + 1]), pack2(xs, xs), pack2(off2, off2)), a, bb);
            } else {
              a = fmaf(x[2 * i], xs, off2);
              bb = fmaf(x[2 * i + 1], xs, off2);
            }
            a = ex2(a);
            bb = ex2(bb);
            ls += a + bb;
            uint32_t h2, l2;
            split_weights(a, bb, h2, l2);
            if (i & 1) {
              ph[i >> 1] |= h2 << 16;
              pl[i >> 1] |= l2 << 16;
            } else {
              ph[i >> 1] = h2;
              pl[i >> 1] = l2;
            }
          }
          const float es = block_scale(e, m_new);
          if constexpr (SCL) ls *= ex2(-lv);  // the weights without the scale
          ls *= exp2_int(es);
          // P^T operand: row r, keys [16 qtr, +16) = one core-matrix row
          unsigned char* pbuf = sm + kOffP + pb * (NAR ? nar_p_buf(nar) : kPBuf);
          const int off = core_off(r, 16 * qtr, kT);
          *reinterpret_cast<uint4*>(pbuf + off) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
          *reinterpret_cast<uint4*>(pbuf + (NAR ? core_off(nar, 0, kT) : kPHalf) + off) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
          // its block's scale: sub 0 that of the high terms, sub 1 that of the low
          // ones: the row's bytes [hi 0, hi 1, lo 0, lo 1], or NAR two rows' [0, 1]
          const int n = NAR ? r + sub * nar : r;
          st_shared_u8(sbase + kOffSf + 512 * pb + 16 * (n & 31) + 4 * (n >> 5) + (NAR ? 0 : 2 * sub) + kh,
                       scale_byte(es) - sub * kLoShift);
        }
        // then the rows that moved (P V(cur - 1) has to be in O^T first; the
        // wait overlaps the work above)
        if (any) {
          const int xp = cur - 1;
          if (!wait_or_fail(kBarPFree + xp % kPBufs, (xp / kPBufs) & 1, 1024)) continue;
          tc_fence_after();
          // the factors of rows [0, 32) and [32, 64), four to a load; a half in
          // which no row moved stays as it is
#pragma unroll 1
          for (int half = 0; half < (NAR ? nar >> 4 : 2); ++half) {
            if (!__any_sync(0xffffffffu, al[32 * half + lane] != 1.f)) continue;
            const float4* af = reinterpret_cast<const float4*>(al + 32 * half);
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
              uint32_t o[32];
              const uint32_t ta = tmem + lane_base + kColO + 64 * (2 * kh + k) + 32 * half;
              tmem_ld_32x32b_x32(ta, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 f = af[i];
                o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * f.x);
                o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * f.y);
                o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * f.z);
                o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * f.w);
              }
              tmem_st_32x32b_x32(ta, o);
            }
          }
          tmem_wait_st();
        }
        l = l * alpha + ls;
        m_ref = m_new;
        // latent rows past S in the item's last tile (a partial page, pages
        // never loaded) are zeroed so that 0 * garbage cannot reach O; Q K^T
        // of this tile has completed (S was full)
        const int zt0 = (lt == pc.nt - 1 && (pc.S % kT) != 0) ? pc.S - lt * kT : kT;
        if (zt0 < kT) {
          unsigned char* vst = sm + (cur % kSlots) * kTileBytes;
          for (int idx = tid - 128; idx < (kT - zt0) * kChunks * 8; idx += kSoftmaxThreads) {
            const int row = zt0 + idx / (kChunks * 8);
            const int rem = idx % (kChunks * 8);
            *reinterpret_cast<uint4*>(vst + (rem >> 3) * kRegion + row * 128 + (rem & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
        }
        tc_fence_before();  // the O^T rescale, before the arrive
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + pb));
      }

      // -- epilogue: this thread's lane holds latent column 128 a + 32 q + lane
      // of chunks a = 2 kh, 2 kh + 1, for all packed rows (the TMEM columns).
      // Every piece leaves (m, l) and its unnormalised O^T in groups of four
      // rows, partial[piece][row / 4][column][row % 4] (mla_acc_index): a
      // lane's four rows are one 16-byte store and a warp's stores of a group
      // are 512 contiguous bytes. The merge kernel writes the output rows.
      // The row sum does not depend on O: its exchange overlaps the last P V.
      const float lrow = exchange(l, false);
      wait_or_fail(kBarOFull, piece_idx & 1, 4096);
      tc_fence_after();
      ++piece_idx;
      if (!ok) continue;
      const int64_t piece = (int64_t)pc.j + c;
      const int ldr = mla_row_stride(p.max_rows);
#pragma unroll 1
      for (int k = 0; k < (NAR ? 2 : 4); ++k) {
        const int a = 2 * kh + (NAR ? k : k >> 1);
        const int r0 = NAR ? 0 : 32 * (k & 1);
        if (r0 >= pc.R) continue;  // warp-uniform
        uint32_t o[32];
        tmem_ld_32x32b_x32(tmem + lane_base + kColO + 64 * a + r0, o);
        if constexpr (NAR) {
          uint32_t lo[32];
          tmem_ld_32x32b_x32(tmem + lane_base + kColO + 64 * a + nar, lo);
          tmem_wait_ld();
#pragma unroll
          for (int w = 0; w < 32; ++w) o[w] = __float_as_uint(__uint_as_float(o[w]) + __uint_as_float(lo[w]));
        } else {
          tmem_wait_ld();
        }
        const int col = 128 * a + 32 * q + lane;
        const int nrow = ldr - r0 < 32 ? ldr - r0 : 32;
        if constexpr (CLU) {
#pragma unroll
          for (int w = 0; w < 32; ++w)
            if (r0 + w < pc.R) part[(r0 + w) * kMlaNope + col] = __uint_as_float(o[w]);
          continue;
        }
#pragma unroll
        for (int w = 0; w < 8; ++w)
          if (4 * w < nrow)
            *reinterpret_cast<float4*>(p.ws_acc + mla_acc_index(piece, r0 + 4 * w, col, ldr)) =
                make_float4(__uint_as_float(o[4 * w]), __uint_as_float(o[4 * w + 1]),
                            __uint_as_float(o[4 * w + 2]), __uint_as_float(o[4 * w + 3]));
      }
      if (CLU) {
        if (row_ok && kh == 0 && sub == 0) {
          part_ml[2 * r] = m_ref;
          part_ml[2 * r + 1] = lrow;
        }
      } else if (row_ok && kh == 0 && sub == 0) {
        p.ws_ml[(piece * p.max_rows + r) * 2 + 0] = m_ref;
        p.ws_ml[(piece * p.max_rows + r) * 2 + 1] = lrow;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOFree));
    }
  }

  if constexpr (CLU) {
    __syncwarp();
    cluster_arrive();  // behind this thread's part of the partial
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  if constexpr (CLU) {
    __syncwarp();
    join_cluster<kThreads, kMlaNope>(p, j_first, meta, c & (p.cluster - 1), smem_addr(part), kMlaNope,
                                     smem_addr(part_ml));
  }
}

using Kernel = void (*)(const Params, const CUtensorMap, const CUtensorMap);
Kernel pick(const Params& p) {
  const bool nar = p.max_rows <= kNarRows;
  if (p.cluster > 0) return nar ? va_mla_tc_kernel<true, true, true> : va_mla_tc_kernel<true, true, false>;
  if (p.k_scales) return nar ? va_mla_tc_kernel<true, false, true> : va_mla_tc_kernel<true, false, false>;
  return va_mla_tc_kernel<false, false, false>;
}

}  // namespace

void mla_tc_clusters(int32_t* caps) {
  // one CTA an SM in either form
  cluster_caps(va_mla_tc_kernel<true, true, false>, kThreads, kSmemBytes + 1024, caps);
}

cudaError_t prepare_mla_tc() {
  for (auto fn : {va_mla_tc_kernel<false, false, false>, va_mla_tc_kernel<true, false, false>,
                  va_mla_tc_kernel<true, false, true>, va_mla_tc_kernel<true, true, false>,
                  va_mla_tc_kernel<true, true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes + 1024);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_mla_tc(const Params& p, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe,
                          cudaStream_t stream) {
  // a programmatic dependent of the stream's previous kernel (see the kernel)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.num_splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.cluster > 0) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, pick(p), p, tm_kv, tm_pe);
}

}  // namespace va
