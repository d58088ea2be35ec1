// What the decode kernels over a paged 8-bit cache share: the worker's walk
// over its sequences and their pages, the waits, and the arithmetic of the two
// E4M3/E5M2 terms and of the softmax reference.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace mla {
namespace decode8 {

using namespace sm100;

constexpr int kHeadsPerCta = 64;
constexpr int kDc = 512;
constexpr int kChunk = 8192;              // 64 rows x 128 bytes, 128-byte swizzle
constexpr uint32_t kE5m2A = 1u << 7;      // A's format field: E5M2 (lo) instead of E4M3 (hi)

// The softmax reference r of a row (log2): probabilities are held as 2^(s - r +
// kPScale), and r moves when a tile's maximum leaves [r - kFall, r + kRise].
constexpr float kPScale = 6.75f;
constexpr float kRise = 2.f, kFall = 13.f;   // 2^(6.75 + 2) = 430.5 <= 448
// Where a reference starts above the maximum of the tile that moves it: the
// first one, a higher one (the next are likely lower) and a lower one.  With
// these a maximum that moved it has a power of two as its probability, so a row
// that one key fills is exact.
constexpr float kLeadFirst = 7.75f, kLeadUp = 5.75f, kLeadDown = 8.75f;
constexpr float kTopWindow = 60.f;

// The reference after a tile with maximum mt; `top` is the largest maximum so
// far, this tile's included.
__device__ __forceinline__ float next_reference(float ref, float mt, float top) {
  const float to = fmaxf(mt, top - kTopWindow);
  return to > ref + kRise ? to + kLeadUp : to < ref - kFall ? to + kLeadDown : ref;
}

// Warp-uniform bounded wait (all lanes poll; lane 0 owns the limit).
__device__ __forceinline__ bool wait_w(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                       uint64_t limit = kWaitLimitCycles) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  const uint64_t t0 = sm_cycles();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_for(bar, parity, 20000))) return true;
    {
      int give_up = 0;
      if ((threadIdx.x & 31) == 0) give_up = (*abort_flag != 0) || (sm_cycles() - t0 > limit);
      if (__shfl_sync(0xffffffffu, give_up, 0)) return false;
    }
  }
}

// The sequences whose tiles lie in this worker's range of work units (as in
// tile_deal.cuh, for any batch size): every role walks them by itself from the
// first one, whose number and unit prefix the block finds together.
struct Segments {
  const int32_t* seqlens;
  int B, b;             // b: the sequence after the current one
  int64_t cap, pre, u0, u1;
  int32_t len_b;        // its length, read ahead
  int cur;              // the current sequence, its tiles [lo, hi) and length
  int64_t lo, hi, L;
  __device__ bool next() {
    while (b < B && pre < u1) {
      cur = b++;
      L = clamp_len(len_b, cap);
      if (b < B) len_b = seqlens[b];
      const int64_t nt = tiles_of(L), r0 = pre + kSwitchUnits;
      if (nt == 0) continue;
      pre = r0 + nt;
      lo = max(r0, u0) - r0;
      hi = min(r0 + nt, u1) - r0;
      if (lo < hi) return true;
    }
    return false;
  }
};

// All threads, with len0 = seqlens[threadIdx.x]; `scratch` is shared memory for kThreads / 32 + 3 values.  False
// if the worker has no units.
template <int kThreads>
__device__ __forceinline__ bool find_segments(int32_t len0, const int32_t* seqlens, int B,
                                              int64_t cap, int w, int W, int64_t* scratch,
                                              Segments* out) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t sum = units_of(clamp_len(len0, cap));
  for (int b = threadIdx.x + kThreads; b < B; b += kThreads)
    sum += units_of(clamp_len(seqlens[b], cap));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scratch[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) total += scratch[k];
  __syncthreads();
  // (A 64-bit division is a long subroutine; both are needed at once here.)
  const bool small = total * W <= int64_t(UINT32_MAX);
  const int64_t u0 = small ? int64_t(uint32_t(w) * uint32_t(total) / uint32_t(W))
                           : worker_tile_begin(w, total, W);
  const int64_t u1 = small ? int64_t(uint32_t(w + 1) * uint32_t(total) / uint32_t(W))
                           : worker_tile_begin(w + 1, total, W);
  if (u0 >= u1) return false;
  // The sequence that unit u0 belongs to, kThreads of them at a time.
  int64_t base = 0;
#pragma unroll 1
  for (int b0 = 0;; b0 += kThreads) {
    const int b = b0 + int(threadIdx.x);
    const int32_t len = b0 == 0 ? len0 : b < B ? seqlens[b] : 0;
    const int64_t n = b < B ? units_of(clamp_len(len, cap)) : 0;
    int64_t e = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) e += u;
    }
    if (lane == 31) scratch[warp] = e;
    __syncthreads();
    int64_t chunk = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) e += scratch[k];
      chunk += scratch[k];
    }
    e += base;
    if (u0 < e && u0 >= e - n)
      scratch[kWarps] = b, scratch[kWarps + 1] = e - n, scratch[kWarps + 2] = len;
    __syncthreads();
    base += chunk;
    // Some chunk holds u0 < total, unless a length has changed since it was counted (by a
    // call on another stream that should have been ordered): then the walk ends here.
    if (u0 < base || b0 + kThreads >= B) break;
  }
  *out = Segments{seqlens, B,  int(scratch[kWarps]),         cap, scratch[kWarps + 1],
                  u0,      u1, int32_t(scratch[kWarps + 2]), 0,   0,
                  0,       0};
  __syncthreads();             // before the scratch is used for anything else
  return u0 < base;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 32 scores to probabilities p = 2^(s f + shift), each split into hi (E4M3) + lo
// (E5M2) through fp16; returns their sum.
__device__ __forceinline__ float split_probabilities(const uint32_t (&x)[32], float f, float shift,
                                                     uint32_t (&hi8)[8], uint32_t (&lo8)[8]) {
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t h[2], l[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 z = fma2(make_float2(__uint_as_float(x[4 * j + 2 * e]),
                                        __uint_as_float(x[4 * j + 2 * e + 1])),
                            make_float2(f, f), make_float2(shift, shift));
      const float2 p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
      sum = add2(sum, p);
      const __half2 p16 = __floats2half2_rn(p.x, p.y);
      h[e] = __nv_cvt_halfraw2_to_fp8x2(p16, __NV_SATFINITE, __NV_E4M3);
      const __half2 back(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(h[e]), __NV_E4M3));
      l[e] = __nv_cvt_halfraw2_to_fp8x2(__hsub2(p16, back), __NV_SATFINITE, __NV_E5M2);
    }
    hi8[j] = h[0] | (h[1] << 16);
    lo8[j] = l[0] | (l[1] << 16);
  }
  return sum.x + sum.y;
}

// The power of two 2^k that a query row is held in units of follows its latent
// part, but no further down than where fp32 holds everything made of it: the
// scaled rotary part stays below 2^(kRopeLead + 9), so that its products with
// keys in units of a page scale of 2^-40 are finite, and 2^k times such a scale
// and the softmax scale stays a normal number.  A row whose latent part is zero, or
// 2^kRopeLead times smaller than its rotary part, or below 2^-51, is held in
// larger units than its latent part needs, which then loses at most 2^-10 of a
// unit: 2^-57 of the rotary part's largest value, or 2^-70.
constexpr int kRopeLead = 40, kMinQueryExp = -60;

// What the rotary part's largest magnitude (its bf16 bits) counts for beside the
// latent part's: 2^-kRopeLead of itself, in bits.
__device__ __forceinline__ uint32_t rope_magnitude(uint32_t top) {
  constexpr uint32_t lead = uint32_t(kRopeLead) << 7;
  return top > lead ? top - lead : 0u;
}
// Exponent of a row whose largest bf16 magnitude has the bits `top`: the smallest k with
// top <= 448 * 2^k = 1.75 * 2^(8 + k) (top = m 2^(e - 127), 7 mantissa bits, m <= 1.75
// up to 96 / 128), within [kMinQueryExp, 120].
__device__ __forceinline__ int query_exponent(uint32_t top) {
  return min(max(int(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 96u), kMinQueryExp), 120);
}
// log2 of the scores' factor: never 0, so that a masked key's -inf stays -inf (scores
// that a smaller factor would make are 0 beside any other).
__device__ __forceinline__ float score_factor(float row_scale, float page_scale) {
  return fmaxf(row_scale * page_scale, 1.17549435e-38f);
}
__device__ __forceinline__ float exp2i(int k) { return __uint_as_float(uint32_t(127 + k) << 23); }

// The larger of each half of two words of bf16 magnitudes (sign bits cleared), and
// the larger half of one.
__device__ __forceinline__ uint32_t max_magnitude2(uint32_t top2, uint32_t w) {
  return __vmaxu2(top2, w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t larger_half(uint32_t top2) {
  return max(top2 & 0xFFFFu, top2 >> 16);
}

// One word of two bf16 values times the power of two inv2 (bf16 in both halves:
// exact), as two E4M3 terms of two codes each, through fp16 (exact down to 2^-14).
__device__ __forceinline__ void split_query(uint32_t w, __nv_bfloat162 inv2, uint32_t* hi,
                                            uint32_t* lo) {
  const __nv_bfloat162 s = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), inv2);
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&s);
  const __half2 x = __floats2half2_rn(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u));
  *hi = __nv_cvt_halfraw2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
  const __half2 back(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(*hi), __NV_E4M3));
  *lo = __nv_cvt_halfraw2_to_fp8x2(__hsub2(x, back), __NV_SATFINITE, __NV_E4M3);
}
// The RoPE part of a query row in the same units.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, __nv_bfloat162 inv2) {
  const __nv_bfloat162 s = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), inv2);
  return *reinterpret_cast<const uint32_t*>(&s);
}

// This CTA's share of the queries into L2, before the lengths say which of them
// it needs (one thread): all CTAs together ask for each row once, and the first
// query block is then read from L2 instead of from memory behind a TLB miss.
__device__ __forceinline__ void prefetch_queries(const __nv_bfloat16* q_cat, int64_t bytes,
                                                 int64_t cta, int64_t n_cta) {
  const int64_t share = ((bytes + n_cta - 1) / n_cta + 15) / 16 * 16;
  const int64_t at = cta * share, end = min(at + share, bytes);
  if (at < end)
    bulk_prefetch_l2(reinterpret_cast<const char*>(q_cat) + at, uint32_t(end - at));
}

// The block table into L2 while the lengths are on their way (one warp: at most a
// line a lane, so the first 600 KB of a larger table).
__device__ __forceinline__ void prefetch_table(const PageMap& pm, int B, int64_t cta,
                                               int64_t n_cta) {
  const int64_t line = (threadIdx.x & 31) * n_cta + cta;
  if (line * 128 < int64_t(B) * pm.max_blocks * 4)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(pm.table) + line * 128));
}

// Page rows and scales of a run of tiles: lane l holds tile base + l, and the
// 32 after those are already on their way.
struct PageWalk {
  const PageMap& pm;
  const float* scales;   // or null
  int b, lane;
  int64_t base, hi;
  int64_t row, row_next;
  float sc, sc_next;
  __device__ PageWalk(const PageMap& m, const float* s, int b_, int64_t lo, int64_t hi_)
      : pm(m), scales(s), b(b_), lane(threadIdx.x & 31), base(lo), hi(hi_) {
    fetch(lo, row, sc);
    fetch(lo + 32, row_next, sc_next);
  }
  __device__ void fetch(int64_t t0, int64_t& r, float& s) const {
    const int64_t t = t0 + lane;
    r = t < hi ? pm.tile_row(b, t) : -1;
    s = scales && r >= 0 ? scales[r / kTileKeys] : 1.f;
  }
  // Row (-1: outside the pool) and scale of tile t >= base, the same in all lanes.
  __device__ void at(int64_t t, int64_t* r, float* s) {
    if (t >= base + 32) {
      base += 32;
      row = row_next, sc = sc_next;
      fetch(base + 32, row_next, sc_next);
    }
    *r = __shfl_sync(0xffffffffu, row, int(t - base));
    *s = __shfl_sync(0xffffffffu, sc, int(t - base));
  }
};

// Byte map over the rows of the pool: boxes of 128 codes x 64 rows, 128-byte
// swizzled; rows past the end read as zeros.
inline bool make_code_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes) {
  EncodeTiledFnT fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, cuuint32_t(kTileKeys)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace decode8
}  // namespace mla
