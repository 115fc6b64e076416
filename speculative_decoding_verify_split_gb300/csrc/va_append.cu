// New tokens into the paged KV cache: rotary position embedding of q and k,
// conversion to the cache's type, and the store into the pages that hold the
// tokens' positions, in one launch.
//
//   pairs (x1, x2) of a head's first `rot` columns at position p:
//     y1 = x1 cos(p, i) - x2 sin(p, i),  y2 = x2 cos(p, i) + x1 sin(p, i)
//   stored = y (bf16), or round_e4m3(y / scale), saturating at 448.
//
// Token t of a sequence with L new and S cached tokens (the new ones among
// them) is at position S - L + t. A unit of work is one page of one sequence:
// the (at most 16) new tokens whose positions the page holds. A page belongs
// to one CTA per KV head, so a page's scale (largest |value| over the page's
// tokens) needs no atomics and the results do not depend on the launch order.
// The units of sequence b are numbered from cu[b] / 16 + 2 b: L tokens touch
// at most L / 16 + 2 pages, so the grid needs no device value, and a CTA finds
// its sequence with one pass over cu_seqlens_q (each thread tests its own
// sequences), a single round trip to memory that also brings the lengths.
//
// The products and their difference are rounded separately (no fused
// multiply-add), so the stored bytes are those of the same formula in any
// fp32 arithmetic.
//
// Every byte is read and written once, so the bound is memory: the prompts of
// 8 sequences (14,274 tokens, 32 query and 2 KV heads, page scales, 526 MB)
// take 83.4 us, 93 % of the measured copy bandwidth; latent prompts of 39,119
// tokens (16 query parts, 238 MB) 42.5 us, 82 %: there half the warps' time
// is instruction issue (ncu: 55 % of the issue slots), and the 128-byte query
// parts are stored 1,152 bytes apart. A verify step is latency: the launch and
// two dependent round trips (lengths; page id, rows and table), one more where
// an older token's scale is read: 2.1 us for two sequences, 3.4 us for 64,
// 4.8 us for 256 (1.8 waves of CTAs, half of them without tokens), back to
// back; the call costs the host 3.2 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "va_append.h"
#include "va_fp8.cuh"

namespace va {
namespace {

constexpr int kKvThreads = 128;      // GQA caches: K or V rows of a page and KV head, or query heads
constexpr int kMlaThreads = 256;     // latent caches
// Query heads of a page's tokens per CTA: a warp takes a token's four at a
// time, so four leave no warp a second round (8 / 16 heads: a call of two
// sequences 2.2 -> 2.9 / 3.6 us, prompts of 14K tokens 84 -> 87 us).
constexpr int kHeadsPerCta = 4;
constexpr int kPeHeadsPerCta = 16;   // latent path: 64-wide query parts

// How a cache holds its values.
enum Kind { kBf16 = 0, kE4m3 = 1, kPageScaled = 2 };

// One page of one sequence: tokens at positions [lo, hi) of page pg.
struct Unit {
  int b, tok0;     // sequence; row of the token at position lo
  int64_t pg;      // page index in the sequence
  int64_t lo, hi;
};

struct UnitShared {
  int b, a, L, S;
};

// The unit of this CTA, or false if there is none. Waits for the stream's
// previous kernel, which may write anything read from there on.
template <int NT>
__device__ __forceinline__ bool find_unit(const AppendParams& p, UnitShared* sh, Unit* out) {
  const int64_t u = blockIdx.x;
  // cu[b] lies in [0, total_q], so only these sequences can hold unit u: few
  // of a batch of short ones
  const int64_t slack = p.total_q / kPageSize;
  const int b0 = u > slack ? (int)((u - slack - 1) / 2) : 0;
  const int b1 = u / 2 + 1 < p.num_seqs ? (int)(u / 2 + 1) : p.num_seqs;
  auto holds = [&](int b, int a, int e) {
    const int64_t g0 = (int64_t)(a / kPageSize) + 2 * (int64_t)b;
    const int64_t g1 = (int64_t)(e / kPageSize) + 2 * ((int64_t)b + 1);
    return a >= 0 && g0 <= u && u < g1;
  };
  int b, a, L;
  int64_t S;
  if (b1 - b0 <= 32) {
    // one sequence a lane: every warp finds the unit for itself
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    b = b0 + lane;
    int e = 0, s = 0;
    a = -1;
    if (b < b1) {
      a = p.cu_q[b];
      e = p.cu_q[b + 1];
      s = p.seqused_k[b];
    }
    const unsigned who = __ballot_sync(0xffffffffu, b < b1 && holds(b, a, e));
    if (who == 0) return false;
    const int src = __ffs((int)who) - 1;
    b = b0 + src;
    a = __shfl_sync(0xffffffffu, a, src);
    L = __shfl_sync(0xffffffffu, e, src) - a;
    S = __shfl_sync(0xffffffffu, s, src);
  } else {
    if (threadIdx.x == 0) sh->b = -1;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int j = b0 + threadIdx.x; j < b1; j += NT) {
      const int ja = p.cu_q[j], je = p.cu_q[j + 1], js = p.seqused_k[j];
      if (holds(j, ja, je)) {
        sh->b = j;
        sh->a = ja;
        sh->L = je - ja;
        sh->S = js;
      }
    }
    __syncthreads();
    b = sh->b;
    if (b < 0) return false;
    a = sh->a;
    L = sh->L;
    S = sh->S;
  }
  // (prefix sums that decrease may name a unit twice: whatever was found, the
  // rows stay inside the tensors)
  L = L < p.total_q - a ? L : p.total_q - a;
  if (L <= 0) return false;
  const int64_t pos0 = S - L;
  const int64_t first = pos0 > 0 ? pos0 : 0;  // tokens before position 0 have no place
  const int64_t i = u - ((int64_t)(a / kPageSize) + 2 * (int64_t)b);
  out->b = b;
  out->pg = first / kPageSize + i;
  const int64_t pa = out->pg * kPageSize, pe = pa + kPageSize;
  out->lo = pa > first ? pa : first;
  out->hi = pe < S ? pe : S;
  out->tok0 = a + (int)(out->lo - pos0);
  return out->lo < out->hi;
}

// Row of the cos | sin table of token row tok at position x.
__device__ __forceinline__ const float* table_row(const AppendParams& p, int tok, int64_t x) {
  if (p.positions) x = p.positions[tok];
  x = x < 0 ? 0 : (x >= p.max_pos ? p.max_pos - 1 : x);
  return p.cos_sin + x * p.cs_s0;
}

__device__ __forceinline__ void unpack4(uint2 w, float* x) {
  x[0] = __uint_as_float(w.x << 16);
  x[1] = __uint_as_float(w.x & 0xFFFF0000u);
  x[2] = __uint_as_float(w.y << 16);
  x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s), every operation rounded by itself.
__device__ __forceinline__ void rotate(float& x1, float& x2, float c, float s) {
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  const float y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1;
  x2 = y2;
}

// Where a lane's eight columns of a 256-wide head lie: two groups of four at
// o1 and o2. Halves: rotated lanes hold pairs (4 l + i, rot / 2 + 4 l + i),
// the others the columns past `rot` in order. Interleaved: eight columns in a
// row, pairs (2 i, 2 i + 1).
struct Lane {
  int o1, o2;
  bool turn;  // these columns are rotated
};

template <bool INTER>
__device__ __forceinline__ Lane lane_columns(int lane, int rot) {
  Lane c;
  if (INTER) {
    c.o1 = 8 * lane;
    c.o2 = c.o1 + 4;
    c.turn = c.o1 < rot;
  } else {
    const int half = rot / 2;
    c.turn = 4 * lane < half;
    c.o1 = c.turn ? 4 * lane : rot + 2 * (4 * lane - half);
    c.o2 = c.turn ? half + 4 * lane : c.o1 + 4;
  }
  return c;
}

template <bool INTER>
__device__ __forceinline__ void rotate8(float* x, float4 c, float4 s) {
  if (INTER) {
    rotate(x[0], x[1], c.x, s.x);
    rotate(x[2], x[3], c.y, s.y);
    rotate(x[4], x[5], c.z, s.z);
    rotate(x[6], x[7], c.w, s.w);
  } else {
    rotate(x[0], x[4], c.x, s.x);
    rotate(x[1], x[5], c.y, s.y);
    rotate(x[2], x[6], c.z, s.z);
    rotate(x[3], x[7], c.w, s.w);
  }
}

__device__ __forceinline__ uint2 to_bf16x4(const float* x) {
  return make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// x / scale. By a power of two in [2^-64, 2^64] the quotient is the product
// with the (exact) reciprocal.
struct Divisor {
  float scale, inv;
  bool power;
  __device__ __forceinline__ explicit Divisor(float s) : scale(s) {
    const uint32_t b = __float_as_uint(s);
    power = (b & 0x807FFFFFu) == 0 && b >= (63u << 23) && b <= (191u << 23);
    inv = __uint_as_float((254u << 23) - b);  // 2^-e of 2^e
  }
  __device__ __forceinline__ void divide8(float* x) const {
    if (power) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], inv);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], scale);
    }
  }
};

__device__ __forceinline__ uint32_t pack_e4m3x4(const float* x) {
  return pack_fp8x2(x[0], x[1]) | (pack_fp8x2(x[2], x[3]) << 16);
}

// Eight codes under scale `had` as codes under scale `now`.
__device__ __forceinline__ uint2 rescale8(uint2 w, float had, const Divisor& now) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_fp8x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)) & 0xFFFFu);
    x[2 * i] = __fmul_rn(f.x, had);
    x[2 * i + 1] = __fmul_rn(f.y, had);
  }
  now.divide8(x);
  return make_uint2(pack_e4m3x4(x), pack_e4m3x4(x + 4));
}

// A page scale as it is read: finite and positive.
__device__ __forceinline__ float usable_scale(float s) {
  return fminf(fmaxf(s, kMinPageScale), kMaxPageScale);  // NaN -> the smallest
}

// The smallest 2^e, -64 <= e <= 64, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -64 ? -64 : (e > 64 ? 64 : e);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// The largest |value| of eight bf16 ones, in pairs; NaN loses against a number.
__device__ __forceinline__ float amax8(uint4 w) {
  auto pair = [](uint32_t v) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)); };
  const __nv_bfloat162 m = __hmax2(__hmax2(pair(w.x), pair(w.y)), __hmax2(pair(w.z), pair(w.w)));
  return fmaxf(__low2float(m), __high2float(m));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---- keys, values and queries of a GQA cache -----------------------------------
//
// blockIdx.y < 2 hkv: the page's K rows (even) or V rows (odd) of one KV head,
// four slots of the page per warp. Above: the same tokens' rows of
// kHeadsPerCta query heads, a token per warp.
template <int KIND, bool INTER>
__global__ void __launch_bounds__(kKvThreads, 8) va_append_kernel(const AppendParams p) {
  constexpr int kWarps = kKvThreads / 32;
  __shared__ UnitShared sh;
  __shared__ float s_amax[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Unit u;
  if (!find_unit<kKvThreads>(p, &sh, &u)) return;  // CTA-uniform
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lane col = lane_columns<INTER>(lane, p.rot);

  if ((int)blockIdx.y >= 2 * p.hkv) {  // ---- query heads
    const int hb = ((int)blockIdx.y - 2 * p.hkv) * kHeadsPerCta;
    for (int t = warp; t < (int)(u.hi - u.lo); t += kWarps) {  // a token's heads, all their loads at once
      const int tok = u.tok0 + t;
      const uint16_t* src = p.q + (int64_t)tok * p.q_s0;
      uint2 w1[kHeadsPerCta], w2[kHeadsPerCta];
#pragma unroll
      for (int i = 0; i < kHeadsPerCta; ++i) {
        const uint16_t* row = src + (int64_t)(hb + i) * p.q_s1;
        const bool on = hb + i < p.hq;
        w1[i] = on ? *reinterpret_cast<const uint2*>(row + col.o1) : make_uint2(0, 0);
        w2[i] = on ? *reinterpret_cast<const uint2*>(row + col.o2) : make_uint2(0, 0);
      }
      float4 c = make_float4(0.f, 0.f, 0.f, 0.f), sn = c;
      if (col.turn) {
        const float* cs = table_row(p, tok, u.lo + t) + 4 * lane;
        c = *reinterpret_cast<const float4*>(cs);
        sn = *reinterpret_cast<const float4*>(cs + p.rot / 2);
      }
      uint16_t* out = p.q_out + (int64_t)tok * p.qo_s0;
#pragma unroll
      for (int i = 0; i < kHeadsPerCta; ++i) {
        float x[8];
        unpack4(w1[i], x);
        unpack4(w2[i], x + 4);
        if (col.turn) rotate8<INTER>(x, c, sn);
        if (hb + i < p.hq) {
          uint16_t* dst = out + (int64_t)(hb + i) * p.qo_s1;
          *reinterpret_cast<uint2*>(dst + col.o1) = to_bf16x4(x);
          *reinterpret_cast<uint2*>(dst + col.o2) = to_bf16x4(x + 4);
        }
      }
    }
    return;
  }

  // ---- K or V of one KV head of the page
  const int h = (int)blockIdx.y >> 1;
  if (u.pg >= p.bt_width) return;
  // the page id and the new rows are read together
  const int page = p.block_table[(int64_t)u.b * p.bt_s0 + u.pg * p.bt_s1];
  const bool is_k = (blockIdx.y & 1) == 0;
  const int s_lo = (int)(u.lo - u.pg * kPageSize), s_hi = (int)(u.hi - u.pg * kPageSize);
  const uint16_t* src = (is_k ? p.k + (int64_t)h * p.k_s1 : p.v + (int64_t)h * p.v_s1);
  const int64_t src_s0 = is_k ? p.k_s0 : p.v_s0;
  const CacheView& c = is_k ? p.kc : p.vc;
  const float* descale = is_k ? p.k_descale : p.v_descale;
  float scale = 1.f;
  const bool divide = KIND != kPageScaled && descale != nullptr;
  if (divide) scale = *descale;

  // the four slots' loads go out together
  uint2 w1[4], w2[4];
  float4 cs[4], sn[4];
  const bool turn = is_k && col.turn;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int s = warp + kWarps * k;
    const bool on = s >= s_lo && s < s_hi;
    const uint16_t* row = src + (int64_t)(u.tok0 + s - s_lo) * src_s0;
    w1[k] = on ? *reinterpret_cast<const uint2*>(row + col.o1) : make_uint2(0, 0);
    w2[k] = on ? *reinterpret_cast<const uint2*>(row + col.o2) : make_uint2(0, 0);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int s = warp + kWarps * k;
    cs[k] = sn[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turn && s >= s_lo && s < s_hi) {
      const float* row = table_row(p, u.tok0 + s - s_lo, u.pg * kPageSize + s) + 4 * lane;
      cs[k] = *reinterpret_cast<const float4*>(row);
      sn[k] = *reinterpret_cast<const float4*>(row + p.rot / 2);
    }
  }
  if ((unsigned)page >= (unsigned)p.num_blocks) return;
  const int64_t base = (int64_t)page * c.s0 + (int64_t)h * c.s2;
  // older tokens of the page: their scale, and their codes in case it grows
  float had = 0.f;
  uint2 old[4];
  if (KIND == kPageScaled && s_lo > 0) {
    had = c.scales[(int64_t)page * c.sc_s0 + (int64_t)h * c.sc_s1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = warp + kWarps * k;
      const unsigned char* row = static_cast<unsigned char*>(c.data) + base + (int64_t)s * c.s1;
      old[k] = make_uint2(0, 0);
      if (s < s_lo)
        old[k] = make_uint2(*reinterpret_cast<const uint32_t*>(row + col.o1),
                            *reinterpret_cast<const uint32_t*>(row + col.o2));
    }
  }
  float x[4][8];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    unpack4(w1[k], x[k]);
    unpack4(w2[k], x[k] + 4);
    if (turn) rotate8<INTER>(x[k], cs[k], sn[k]);
    if (KIND == kPageScaled) {
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[k][i]));  // NaN counts as 0
    }
  }
  if (KIND == kPageScaled) {
    amax = warp_max(amax);
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();  // every thread has read the old scale, too
    amax = fmaxf(fmaxf(s_amax[0], s_amax[1]), fmaxf(s_amax[2], s_amax[3]));
    scale = scale_for(amax);
    if (s_lo > 0) {  // the page's older tokens keep their scale, or are rounded to the larger one
      had = usable_scale(had);
      scale = fmaxf(scale, had);
      if (scale > had) {
        unsigned char* dst = static_cast<unsigned char*>(c.data) + base;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int s = warp + kWarps * k;
          if (s >= s_lo) continue;
          const uint2 now = rescale8(old[k], had, Divisor(scale));
          *reinterpret_cast<uint32_t*>(dst + (int64_t)s * c.s1 + col.o1) = now.x;
          *reinterpret_cast<uint32_t*>(dst + (int64_t)s * c.s1 + col.o2) = now.y;
        }
      }
    }
    if (threadIdx.x == 0) c.scales[(int64_t)page * c.sc_s0 + (int64_t)h * c.sc_s1] = scale;
  }
  const Divisor by(scale);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int s = warp + kWarps * k;
    if (s < s_lo || s >= s_hi) continue;
    if (KIND == kPageScaled || divide) by.divide8(x[k]);
    if (KIND == kBf16) {
      uint16_t* dst = static_cast<uint16_t*>(c.data) + base + (int64_t)s * c.s1;
      *reinterpret_cast<uint2*>(dst + col.o1) = to_bf16x4(x[k]);
      *reinterpret_cast<uint2*>(dst + col.o2) = to_bf16x4(x[k] + 4);
    } else {
      unsigned char* dst = static_cast<unsigned char*>(c.data) + base + (int64_t)s * c.s1;
      *reinterpret_cast<uint32_t*>(dst + col.o1) = pack_e4m3x4(x[k]);
      *reinterpret_cast<uint32_t*>(dst + col.o2) = pack_e4m3x4(x[k] + 4);
    }
  }
}

// ---- rows of a latent cache ------------------------------------------------------
//
// blockIdx.y == 0: the page's rows [latent 512 | rope 64], two slots per
// warp; a lane holds latent columns 8 l.. and 256 + 8 l.. and one rope pair.
// Above: the tokens' 64-wide rope parts of kPeHeadsPerCta query heads, eight
// lanes a row.
template <int KIND, bool INTER>
__global__ void __launch_bounds__(kMlaThreads, 4) va_append_mla_kernel(const AppendParams p) {
  constexpr int kWarps = kMlaThreads / 32;
  __shared__ UnitShared sh;
  __shared__ float s_amax[kWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Unit u;
  if (!find_unit<kMlaThreads>(p, &sh, &u)) return;  // CTA-uniform
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (blockIdx.y > 0) {  // ---- query heads
    const int h0 = ((int)blockIdx.y - 1) * kPeHeadsPerCta;
    const int nh = p.hq - h0 < kPeHeadsPerCta ? p.hq - h0 : kPeHeadsPerCta;
    const int l8 = lane & 7, g = lane >> 3;
    const int o1 = INTER ? 8 * l8 : 4 * l8, o2 = INTER ? o1 + 4 : 32 + o1;
    for (int t = warp; t < (int)(u.hi - u.lo); t += kWarps) {  // a token's heads g, g + 4, .., all loads at once
      const int tok = u.tok0 + t;
      const uint16_t* src = p.q + (int64_t)tok * p.q_s0;
      uint2 w1[kPeHeadsPerCta / 4], w2[kPeHeadsPerCta / 4];
#pragma unroll
      for (int i = 0; i < kPeHeadsPerCta / 4; ++i) {
        const bool on = g + 4 * i < nh;
        const uint16_t* row = src + (int64_t)(h0 + g + 4 * i) * p.q_s1;
        w1[i] = on ? *reinterpret_cast<const uint2*>(row + o1) : make_uint2(0, 0);
        w2[i] = on ? *reinterpret_cast<const uint2*>(row + o2) : make_uint2(0, 0);
      }
      const float* cs = table_row(p, tok, u.lo + t) + 4 * l8;
      const float4 c = *reinterpret_cast<const float4*>(cs);
      const float4 sn = *reinterpret_cast<const float4*>(cs + kMlaPe / 2);
      uint16_t* out = p.q_out + (int64_t)tok * p.qo_s0;
#pragma unroll
      for (int i = 0; i < kPeHeadsPerCta / 4; ++i) {
        float x[8];
        unpack4(w1[i], x);
        unpack4(w2[i], x + 4);
        rotate8<INTER>(x, c, sn);
        if (g + 4 * i < nh) {
          uint16_t* dst = out + (int64_t)(h0 + g + 4 * i) * p.qo_s1;
          *reinterpret_cast<uint2*>(dst + o1) = to_bf16x4(x);
          *reinterpret_cast<uint2*>(dst + o2) = to_bf16x4(x + 4);
        }
      }
    }
    return;
  }

  if (u.pg >= p.bt_width) return;
  // the page id and the new rows are read together
  const int page = p.block_table[(int64_t)u.b * p.bt_s0 + u.pg * p.bt_s1];
  const int s_lo = (int)(u.lo - u.pg * kPageSize), s_hi = (int)(u.hi - u.pg * kPageSize);
  const CacheView& c = p.kc;
  float scale = 1.f;
  const bool divide = KIND != kPageScaled && p.k_descale != nullptr;
  if (divide) scale = *p.k_descale;
  // the lane's columns: eight latent ones at n1 and at n2, a rope pair at r1, r2
  const int n1 = 8 * lane, n2 = 256 + 8 * lane;
  const int r1 = INTER ? 2 * lane : lane, r2 = INTER ? r1 + 1 : lane + 32;

  // both slots' loads go out together
  uint4 wa[2], wb[2];
  float y[2][2], cs[2], sn[2];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = warp + kWarps * k;
    const bool on = s >= s_lo && s < s_hi;
    const int tok = u.tok0 + s - s_lo;
    const uint16_t* lat = p.k + (int64_t)tok * p.k_s0;
    const uint16_t* pe = p.v + (int64_t)tok * p.v_s0;
    wa[k] = on ? *reinterpret_cast<const uint4*>(lat + n1) : make_uint4(0, 0, 0, 0);
    wb[k] = on ? *reinterpret_cast<const uint4*>(lat + n2) : make_uint4(0, 0, 0, 0);
    y[k][0] = on ? bf16_bits_to_float(pe[r1]) : 0.f;
    y[k][1] = on ? bf16_bits_to_float(pe[r2]) : 0.f;
    cs[k] = 1.f;
    sn[k] = 0.f;
    if (on && p.cos_sin) {
      const float* row = table_row(p, tok, u.pg * kPageSize + s) + lane;
      cs[k] = row[0];
      sn[k] = row[kMlaPe / 2];
    }
  }
  if ((unsigned)page >= (unsigned)p.num_blocks) return;
  const int64_t base = (int64_t)page * c.s0;
  const float read = KIND == kPageScaled && s_lo > 0 ? c.scales[(int64_t)page * c.sc_s0] : 0.f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (p.cos_sin) rotate(y[k][0], y[k][1], cs[k], sn[k]);
    if (KIND == kPageScaled)  // NaN counts as 0
      amax = fmaxf(fmaxf(amax, fmaxf(amax8(wa[k]), amax8(wb[k]))), fmaxf(fabsf(y[k][0]), fabsf(y[k][1])));
  }
  if (KIND == kPageScaled) {
    amax = warp_max(amax);
    if (lane == 0) s_amax[warp] = amax;
    __syncthreads();  // every thread has read the old scale, too
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, s_amax[w]);
    scale = scale_for(amax);
    if (s_lo > 0) {
      const float had = usable_scale(read);
      scale = fmaxf(scale, had);
      if (scale > had) {
        unsigned char* dst = static_cast<unsigned char*>(c.data) + base;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int s = warp + kWarps * k;
          if (s >= s_lo) continue;
          unsigned char* row = dst + (int64_t)s * c.s1;
          const Divisor now(scale);
          const uint32_t e = (uint32_t)row[kMlaNope + r1] | ((uint32_t)row[kMlaNope + r2] << 8);
          const uint2 a = rescale8(*reinterpret_cast<uint2*>(row + n1), had, now);
          const uint2 b = rescale8(*reinterpret_cast<uint2*>(row + n2), had, now);
          const uint32_t f = rescale8(make_uint2(e, 0), had, now).x;
          *reinterpret_cast<uint2*>(row + n1) = a;
          *reinterpret_cast<uint2*>(row + n2) = b;
          row[kMlaNope + r1] = (unsigned char)f;
          row[kMlaNope + r2] = (unsigned char)(f >> 8);
        }
      }
    }
    if (threadIdx.x == 0) c.scales[(int64_t)page * c.sc_s0] = scale;
  }
  const Divisor by(scale);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int s = warp + kWarps * k;
    if (s < s_lo || s >= s_hi) continue;
    float x[16];
    unpack4(make_uint2(wa[k].x, wa[k].y), x);
    unpack4(make_uint2(wa[k].z, wa[k].w), x + 4);
    unpack4(make_uint2(wb[k].x, wb[k].y), x + 8);
    unpack4(make_uint2(wb[k].z, wb[k].w), x + 12);
    if (KIND == kPageScaled || divide) {
      by.divide8(x);
      by.divide8(x + 8);
      y[k][0] = by.power ? __fmul_rn(y[k][0], by.inv) : __fdiv_rn(y[k][0], scale);
      y[k][1] = by.power ? __fmul_rn(y[k][1], by.inv) : __fdiv_rn(y[k][1], scale);
    }
    if (KIND == kBf16) {
      uint16_t* dst = static_cast<uint16_t*>(c.data) + base + (int64_t)s * c.s1;
      const uint2 a = to_bf16x4(x), b = to_bf16x4(x + 4), d = to_bf16x4(x + 8), e = to_bf16x4(x + 12);
      *reinterpret_cast<uint4*>(dst + n1) = make_uint4(a.x, a.y, b.x, b.y);
      *reinterpret_cast<uint4*>(dst + n2) = make_uint4(d.x, d.y, e.x, e.y);
      dst[kMlaNope + r1] = float_to_bf16_bits(y[k][0]);
      dst[kMlaNope + r2] = float_to_bf16_bits(y[k][1]);
    } else {
      unsigned char* dst = static_cast<unsigned char*>(c.data) + base + (int64_t)s * c.s1;
      *reinterpret_cast<uint2*>(dst + n1) = make_uint2(pack_e4m3x4(x), pack_e4m3x4(x + 4));
      *reinterpret_cast<uint2*>(dst + n2) = make_uint2(pack_e4m3x4(x + 8), pack_e4m3x4(x + 12));
      const uint32_t f = pack_fp8x2(y[k][0], y[k][1]);
      dst[kMlaNope + r1] = (unsigned char)f;
      dst[kMlaNope + r2] = (unsigned char)(f >> 8);
    }
  }
}

using KernelFn = void (*)(const AppendParams);

template <int KIND>
KernelFn pick(bool mla, bool inter) {
  if (mla) return inter ? va_append_mla_kernel<KIND, true> : va_append_mla_kernel<KIND, false>;
  return inter ? va_append_kernel<KIND, true> : va_append_kernel<KIND, false>;
}

}  // namespace

int64_t append_roles(bool mla, const AppendParams& p) {
  const int64_t per = mla ? kPeHeadsPerCta : kHeadsPerCta;
  return (mla ? 1 : 2 * (int64_t)p.hkv) + (p.hq + per - 1) / per;
}

cudaError_t launch_append(const AppendParams& p, bool mla, cudaStream_t stream) {
  const int64_t units = p.total_q / kPageSize + 2 * (int64_t)p.num_seqs;
  const int64_t roles = append_roles(mla, p);
  const KernelFn fn = p.kc.scales ? pick<kPageScaled>(mla, p.interleaved)
                      : p.kc.fp8  ? pick<kE4m3>(mla, p.interleaved)
                                  : pick<kBf16>(mla, p.interleaved);
  // a programmatic dependent of the stream's previous kernel, as the
  // attention kernels are: it touches memory only after that kernel
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)units, (unsigned)roles);
  cfg.blockDim = dim3(mla ? kMlaThreads : kKvThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace va
