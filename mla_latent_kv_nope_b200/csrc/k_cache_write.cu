// Latent rows of many new tokens into a paged cache: the row
//   [RMSNorm(x[0:d_c]) * gamma || RoPE(x[d_c:], position)]
// of each projected token x = W^DKV h, stored in the cache dtype at its slot, or
// as E4M3 codes with one power-of-two scale per page.
#include <cuda_fp8.h>

#include <type_traits>

#include "kernels.h"
#include "rope_table.cuh"
#include "sm100.cuh"

namespace mla {

namespace {

template <typename T, int kVec>
__device__ __forceinline__ void unpack16(const uint4& v, float (&f)[kVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <typename T, int kVec>
__device__ __forceinline__ uint4 pack16(const float (&f)[kVec]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two fp32 products in one instruction.
__device__ __forceinline__ void mul2(float* a, float bx, float by) {
  asm("{\n\t.reg .b64 ra, rb;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "mul.rn.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(a[0]), "+f"(a[1])
      : "f"(bx), "f"(by));
}

__device__ __forceinline__ void load_gamma(const float* gamma, int c, int n, float* g) {
#pragma unroll
  for (int i = 0; i < n; i += 4) {
    const float4 v = gamma ? *reinterpret_cast<const float4*>(gamma + c + i)
                           : make_float4(1.f, 1.f, 1.f, 1.f);
    g[i] = v.x, g[i + 1] = v.y, g[i + 2] = v.z, g[i + 3] = v.w;
  }
}

// The two places of pair k of a d_r-wide rotary block.
__device__ __forceinline__ void pair_at(const mla_rope_table& tab, int d_r, int k, int* i, int* j) {
  const bool inter = tab.layout == MLA_ROPE_INTERLEAVED;
  *i = inter ? 2 * k : k;
  *j = inter ? 2 * k + 1 : k + d_r / 2;
}

// ---------------------------------------------------------------- 16- and 32-bit pages
// One warp per token: the row is read once with 16-byte loads and stays in
// registers (kUnits 16-byte units per lane), the sum of squares is a warp
// reduction, and the row goes out with 16-byte stores.  Bound by HBM (one read
// and one write of the row), for a decode step by latency.  Measured on B200: 8740
// bf16 tokens 5.8 us (3.5 TB/s of 20 MB; 6.4 with the table read at its use), 32
// tokens 2.3 us (2.7).
constexpr int kWriteWarps = 4;

// With kStep a warp more looks whether the step has more tokens than rows (as a
// branch of the one kernel it cost the others 0.15 us at 8740 tokens).
template <typename T, int kUnits, bool kStep>
__global__ void __launch_bounds__(32 * kWriteWarps)
cache_write_kernel(const __grid_constant__ mla_rope_table tab, int rotate,
                   const T* __restrict__ x, int64_t x_stride, const float* __restrict__ gamma,
                   float eps, const int32_t* __restrict__ positions,
                   const int64_t* __restrict__ slots, int T_rows, int d_c, int d_r,
                   int64_t total_rows, T* __restrict__ pool, int* __restrict__ status,
                   const int32_t* __restrict__ planned) {
  constexpr int kVec = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  const int64_t t = int64_t(blockIdx.x) * kWriteWarps + (threadIdx.x >> 5);
  if (kStep && t == T_rows && lane == 0) {
    pdl_wait();
    if (*planned > T_rows) record_status(status, MLA_ERR_BOUNDS);
  }
  if (t >= T_rows) return;
  pdl_wait();
  const T* row = x + t * x_stride;
  uint4 v[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int c = (lane + 32 * u) * kVec;
    v[u] = c < d_c ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
  }
  // Slot, position and rotary pair are asked for before the first use of x (gamma, the
  // same for every token, where the row is stored).
  const int64_t slot = slots[t];
  const int64_t pos = rotate ? positions[t] : 0;
  int pi = lane, pj = lane + d_r / 2;
  if (rotate) pair_at(tab, d_r, lane, &pi, &pj);
  float pa = 0.f, pb = 0.f;
  if (lane < d_r / 2) pa = Storage<T>::to_f(row[d_c + pi]), pb = Storage<T>::to_f(row[d_c + pj]);
  // (Lanes differ in their pair, so the table's read is serialised: while those come.)
  const uint64_t turn = rotate && lane < d_r / 2 ? tab.turn[lane] : 0;
  if (slot < 0) return;               // padding
  if (slot >= total_rows) {
    if (lane == 0) record_status(status, MLA_ERR_BOUNDS);
    return;
  }
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    float f[kVec];
    unpack16<T, kVec>(v[u], f);
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(f[i], f[i], ss);
  }
  const float inv = rsqrtf(warp_sum(ss) / float(d_c) + eps);
  T* dst = pool + slot * (d_c + d_r);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int c = (lane + 32 * u) * kVec;
    if (c < d_c) {
      float f[kVec], g[kVec];
      unpack16<T, kVec>(v[u], f);
      load_gamma(gamma, c, kVec, g);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = f[i] * inv * g[i];
      *reinterpret_cast<uint4*>(dst + c) = pack16<T, kVec>(f);
    }
  }
  for (int k = lane; k < d_r / 2; k += 32) {   // one pair per lane up to d_r = 64
    if (k != lane) {
      pi = k, pj = k + d_r / 2;
      if (rotate) pair_at(tab, d_r, k, &pi, &pj);
      pa = Storage<T>::to_f(row[d_c + pi]), pb = Storage<T>::to_f(row[d_c + pj]);
    }
    if (rotate) {
      float c, s;
      rope_turn_cos_sin(k == lane ? turn : tab.turn[k], pos, tab.amplitude, &c, &s);
      const float a = pa, b = pb;
      pa = a * c - b * s;
      pb = a * s + b * c;
    }
    dst[d_c + pi] = Storage<T>::from_f(pa);
    dst[d_c + pj] = Storage<T>::from_f(pb);
  }
}

// ---------------------------------------------------------------- 8-bit pages
// One block, or a cluster of two or four that share the rows, per (request, page that
// its new tokens touch).  Bound by latency: the lengths, the page id and the rows, the
// page's maximum, and the arithmetic of a page's rows on one SM, which is why the page
// is shared.  The rows are copied to shared memory asynchronously (one read of x, all
// in flight at once; held in registers, a block filled an SM and 150 pages took two
// waves), each warp norms its own, the page's largest magnitude is reduced over the
// block and the cluster, the new exponent fixed, and the codes written.  Measured on
// B200: 64 tokens, one a page, 3.7 us; 8740 prompt tokens 8.0 us (9.2 with one block a
// page), 1000 tokens of one prompt 4.7 us (6.8).  If the page held rows before and its
// scale grows, those rows are rescaled first by a power of two, which is exact for the
// rotary keys and for codes that stay normal E4M3 values and rounds the others once more.
constexpr int k8Dc = 512;
constexpr int kMinScaleExp = -40, kMaxScaleExp = 120;

// Smallest k with amax <= 448 * 2^k, within the limits (448 = 0.875 * 2^9).
__device__ __forceinline__ int scale_exponent(float amax) {
  if (!(amax > 0.f)) return kMinScaleExp;
  int e;
  const float f = frexpf(amax, &e);
  const int k = f <= 0.875f ? e - 9 : e - 8;
  return min(max(k, kMinScaleExp), kMaxScaleExp);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t w, float f) {
  const __half2 lo(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xFFFFu), __NV_E4M3));
  const __half2 hi(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> 16), __NV_E4M3));
  return e4m3x4(__low2float(lo) * f, __high2float(lo) * f, __low2float(hi) * f,
                __high2float(hi) * f);
}

template <int kDr, int kSplit>
struct Write8 {
  static constexpr int kRows = kTileKeys / kSplit;             // of a page, a block's
  static constexpr int kThreads = kSplit == 1 ? 512 : 256;
  static constexpr size_t kSmem = size_t(kRows) * 2 * (k8Dc + kDr);
};

template <int kDr, int kSplit>
__global__ void __launch_bounds__(Write8<kDr, kSplit>::kThreads, kSplit == 1 ? 2 : 4)
cache_write8_kernel(const __grid_constant__ mla_rope_table tab, int rotate,
                    const __nv_bfloat16* __restrict__ x, int64_t x_stride, int T_rows,
                    const float* __restrict__ gamma, float eps,
                    const int32_t* __restrict__ query_start, const int32_t* __restrict__ seqlens,
                    int B, int64_t cap, const PageMap pm, uint8_t* __restrict__ pool,
                    float* __restrict__ page_scales, int* __restrict__ status) {
  constexpr int kRowBytes = k8Dc + 2 * kDr, kRows = Write8<kDr, kSplit>::kRows;
  constexpr int k8Threads = Write8<kDr, kSplit>::kThreads, k8Warps = k8Threads / 32;
  extern __shared__ __align__(16) uint8_t s_x[];   // [kRows][d_c + d_r] bf16 as they came
  __shared__ int s_scan[k8Warps];
  __shared__ int s_req, s_first, s_total;
  __shared__ float s_max[k8Warps], s_inv[kRows];
  __shared__ float s_peer[kSplit];                 // each block's largest magnitude
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kSplit > 1 ? int(sm100::cluster_rank()) : 0;
  if (kSplit > 1) sm100::cluster_sync();           // all have started: their shared memory is there
  pdl_wait();

  // The request whose pages cover this block's index: requests are counted
  // blockDim at a time, until the one that passes it (the last block looks at
  // all of them, so that lengths that do not fit are always reported).
  int base = 0;
  const int task = blockIdx.x / kSplit, tasks = int(gridDim.x) / kSplit;
  if (tid == 0) s_req = -1;
  __syncthreads();
  for (int b0 = 0; b0 < B; b0 += k8Threads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < B) {
      const int32_t q0 = query_start[b], q1 = query_start[b + 1], L = seqlens[b];
      const int64_t add = int64_t(q1) - q0;
      if (add < 0 || q0 < 0 || q1 > T_rows || (add > 0 && (L < add || L > cap))) {
        record_status(status, MLA_ERR_BOUNDS);
      } else if (add > 0) {
        n = int((int64_t(L) - 1) / kTileKeys - (L - add) / kTileKeys) + 1;
      }
    }
    int e = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) e += u;
    }
    if (lane == 31) s_scan[warp] = e;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < k8Warps; ++w)
      if (w < warp) e += s_scan[w];
    e += base;
    if (task < e && task >= e - n) s_req = b, s_first = e - n;
    if (tid == k8Threads - 1) s_total = e;
    __syncthreads();
    if (s_req >= 0 && task + 1 < tasks) break;
    base = s_total;
  }
  const int b = s_req;
  if (b < 0) return;
  const int64_t q0 = query_start[b], end = seqlens[b];
  const int64_t start = end - (query_start[b + 1] - q0);        // first new position
  const int64_t j = start / kTileKeys + (task - s_first);       // this page's block
  const int r0 = int(max(start - j * kTileKeys, int64_t(0)));                    // new rows
  const int r1 = int(min(end - j * kTileKeys, int64_t(kTileKeys)));              // [r0, r1)
  const int64_t x0 = q0 + j * kTileKeys - start;                                 // x row of page row 0
  // This block's rows of the page: [p0, p1), new ones [n0, n1).
  const int p0 = rank * kRows, p1 = p0 + kRows, n0 = max(r0, p0), n1 = min(r1, p1);
  // The page id and x are asked for together.
  const int64_t first = pm.tile_row(b, j);

  // Every k8Warps-th new row is this warp's.
  constexpr int kXBytes = 2 * (k8Dc + kDr);
#pragma unroll 1
  for (int r = n0 + warp; r < n1; r += k8Warps) {
    const char* src = reinterpret_cast<const char*>(x + (x0 + r) * x_stride);
    const uint32_t dst = uint32_t(__cvta_generic_to_shared(s_x + (r - p0) * kXBytes));
#pragma unroll
    for (int u = lane; u < kXBytes / 16; u += 32)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + u * 16), "l"(src + u * 16)
                   : "memory");
  }
  float g[16];
  load_gamma(gamma, lane * 8, 8, g);
  load_gamma(gamma, 256 + lane * 8, 8, g + 8);
  // This lane's pair.  (Lanes differ, so the table's read is serialised: while x comes.)
  int ra = lane, rc = lane + kDr / 2;
  const uint64_t turn = kDr > 0 && rotate ? tab.turn[lane] : 0;
  if (kDr > 0 && rotate) pair_at(tab, kDr, lane, &ra, &rc);
  if (first < 0) {
    if (tid == 0) record_status(status, MLA_ERR_BOUNDS);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  uint8_t* page = pool + first * kRowBytes;
  float* page_scale = page_scales + first / kTileKeys;
  const float old_scale = r0 ? *page_scale : 0.f;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  auto row_values = [&](int r, float (&f)[16]) {
    const uint4* row = reinterpret_cast<const uint4*>(s_x + (r - p0) * kXBytes);
    unpack16<__nv_bfloat16, 8>(row[lane], *reinterpret_cast<float(*)[8]>(f));
    unpack16<__nv_bfloat16, 8>(row[lane + 32], *reinterpret_cast<float(*)[8]>(f + 8));
  };
  // The loops over a warp's rows stay rolled: a page is written once, so what
  // its code costs is mostly the fetching of it.
  float amax = 0.f;
#pragma unroll 1
  for (int r = n0 + warp; r < n1; r += k8Warps) {
    float f[16], ss = 0.f;
    row_values(r, f);
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
    const float inv = rsqrtf(warp_sum(ss) * (1.f / k8Dc) + eps);
    float top = 0.f;     // the row's largest |x gamma|; its factor is common and positive
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      mul2(f + e, g[e], g[e + 1]);
      top = fmaxf(top, fmaxf(fabsf(f[e]), fabsf(f[e + 1])));
    }
    amax = fmaxf(amax, top * inv);
    if (lane == 0) s_inv[r - p0] = inv;
  }
  amax = warp_max(amax);
  if (lane == 0) s_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < k8Warps; ++w) amax = fmaxf(amax, s_max[w]);
  if constexpr (kSplit > 1) {
    // Each block tells the others; all have read the page's scale when they meet.
    if (tid < kSplit)
      sm100::st_cluster_u32(sm100::cluster_map(&s_peer[rank], uint32_t(tid)), __float_as_uint(amax));
    sm100::cluster_sync();
#pragma unroll
    for (int w = 0; w < kSplit; ++w) amax = fmaxf(amax, s_peer[w]);
  }
  int k = scale_exponent(amax);
  if (r0 && old_scale > 0.f && old_scale < INFINITY) {
    int e;
    const float f = frexpf(old_scale, &e);
    k = max(k, min(f > 0.5f ? e : e - 1, kMaxScaleExp));
    const float ratio = old_scale * ldexpf(1.f, -k);
    if (ratio != 1.f)
      for (int r = p0 + warp; r < min(r0, p1); r += k8Warps) {
        uint4* row = reinterpret_cast<uint4*>(page + r * kRowBytes);
        uint4 c = row[lane];
        c.x = rescale_e4m3x4(c.x, ratio);
        c.y = rescale_e4m3x4(c.y, ratio);
        c.z = rescale_e4m3x4(c.z, ratio);
        c.w = rescale_e4m3x4(c.w, ratio);
        row[lane] = c;
        if (kDr > 0 && lane < kDr / 8) {
          float f8[8];
          unpack16<__nv_bfloat16, 8>(row[32 + lane], f8);
#pragma unroll
          for (int q = 0; q < 8; ++q) f8[q] *= ratio;
          row[32 + lane] = pack16<__nv_bfloat16, 8>(f8);
        }
      }
  }
  const float inv_scale = ldexpf(1.f, -k);
  if (tid == 0 && rank == 0) *page_scale = ldexpf(1.f, k);
#pragma unroll 1
  for (int r = n0 + warp; r < n1; r += k8Warps) {
    const float inv = s_inv[r - p0] * inv_scale;   // the power of two commutes with the roundings
    uint8_t* row = page + r * kRowBytes;
    float f[16];
    row_values(r, f);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      mul2(f + e, g[e], g[e + 1]);
      mul2(f + e, inv, inv);
    }
    reinterpret_cast<uint2*>(row)[lane] =
        make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
    reinterpret_cast<uint2*>(row)[lane + 32] =
        make_uint2(e4m3x4(f[8], f[9], f[10], f[11]), e4m3x4(f[12], f[13], f[14], f[15]));
    if constexpr (kDr > 0) {
      const __nv_bfloat16* xr = reinterpret_cast<const __nv_bfloat16*>(s_x + (r - p0) * kXBytes) + k8Dc;
      const float a = __bfloat162float(xr[ra]), c = __bfloat162float(xr[rc]);
      float y1 = a, y2 = c;
      if (rotate) {
        float cs, sn;
        rope_turn_cos_sin(turn, j * kTileKeys + r, tab.amplitude, &cs, &sn);
        y1 = a * cs - c * sn;
        y2 = a * sn + c * cs;
      }
      // Rounded to bf16 as in a bf16 cache; the power of two is exact.
      __nv_bfloat16* rope = reinterpret_cast<__nv_bfloat16*>(row + k8Dc);
      rope[ra] = __float2bfloat16_rn(__bfloat162float(__float2bfloat16_rn(y1)) * inv_scale);
      rope[rc] = __float2bfloat16_rn(__bfloat162float(__float2bfloat16_rn(y2)) * inv_scale);
    }
  }
}

}  // namespace

template <typename T>
cudaError_t launch_cache_write(const mla_rope_table* tab, const T* x, int64_t x_stride,
                               const float* gamma, float eps, const int32_t* positions,
                               const int64_t* slots, const int32_t* planned, int T_rows, int d_c,
                               int d_r, int64_t total_rows, T* pool, int* status,
                               cudaStream_t stream) {
  const int64_t warps = int64_t(T_rows) + (planned != nullptr);
  const dim3 grid(unsigned((warps + kWriteWarps - 1) / kWriteWarps)), block(32 * kWriteWarps);
  const mla_rope_table t = tab ? *tab : mla_rope_table{};
  const int units = (d_c * int(sizeof(T)) / 16 + 31) / 32;   // 16-byte units per lane
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, stream, t, int(tab != nullptr), x, x_stride, gamma,
                      eps, positions, slots, T_rows, d_c, d_r, total_rows, pool, status, planned);
  };
  auto pick = [&](auto u) {
    constexpr int kU = decltype(u)::value;
    return planned ? go(cache_write_kernel<T, kU, true>) : go(cache_write_kernel<T, kU, false>);
  };
  if (units <= 1) return pick(std::integral_constant<int, 1>{});
  if (units <= 2) return pick(std::integral_constant<int, 2>{});
  if (units <= 4) return pick(std::integral_constant<int, 4>{});
  return pick(std::integral_constant<int, 8>{});
}

template cudaError_t launch_cache_write<float>(const mla_rope_table*, const float*, int64_t,
                                               const float*, float, const int32_t*,
                                               const int64_t*, const int32_t*, int, int, int,
                                               int64_t, float*, int*, cudaStream_t);
template cudaError_t launch_cache_write<__nv_bfloat16>(const mla_rope_table*, const __nv_bfloat16*,
                                                       int64_t, const float*, float,
                                                       const int32_t*, const int64_t*,
                                                       const int32_t*, int, int, int, int64_t,
                                                       __nv_bfloat16*, int*, cudaStream_t);

cudaError_t launch_cache_write_fp8(const mla_rope_table* tab, const __nv_bfloat16* x,
                                   int64_t x_stride, int T_rows, const float* gamma, float eps,
                                   const int32_t* query_start, const int32_t* seqlens, int B,
                                   int64_t cap, int d_r, const PageMap& pm, uint8_t* pool,
                                   float* page_scales, int* status, int sms,
                                   cudaStream_t stream) {
  const mla_rope_table t = tab ? *tab : mla_rope_table{};
  // A request with n new tokens touches at most min(n, n / 64 + 2) pages.
  const int64_t most = int64_t(T_rows) / kTileKeys + 2 * int64_t(B);
  const int64_t tasks = most < T_rows ? most : T_rows;
  auto go = [&](auto kernel, auto shape) {
    using S = decltype(shape);
    const int split = kTileKeys / S::kRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(tasks * split));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    if constexpr (S::kSmem > 48 * 1024) {   // more than a launch may ask for unannounced
      static bool attr_done[64] = {false};  // of this kernel, by device
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
      if (!attr_done[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
        if (e != cudaSuccess) return e;
        attr_done[dev] = true;
      }
    }
    return cudaLaunchKernelEx(&cfg, kernel, t, int(tab != nullptr), x, x_stride, T_rows, gamma, eps,
                              query_start, seqlens, B, cap, pm, pool, page_scales, status);
  };
  // Blocks to a page.  With a row or two a page there is nothing to share (64 pages:
  // 4.0 us, shared by four blocks 4.5).  Four blocks while all of them run at once: 66
  // pages 5.7 us against 6.0 with two and 6.9 with one, 103 pages 6.7, 7.0 and 7.0,
  // but 168 pages 11.3, 8.0 and 9.2.  Beyond that two blocks keep even with one or ahead
  // (628 pages 22.0 against 23.0, 700 pages of 200 prompts 21.5 against 21.0).
  if (T_rows <= 2 * int64_t(B))
    return d_r ? go(cache_write8_kernel<64, 1>, Write8<64, 1>{})
               : go(cache_write8_kernel<0, 1>, Write8<0, 1>{});
  if (4 * tasks <= 3 * int64_t(sms))
    return d_r ? go(cache_write8_kernel<64, 4>, Write8<64, 4>{})
               : go(cache_write8_kernel<0, 4>, Write8<0, 4>{});
  return d_r ? go(cache_write8_kernel<64, 2>, Write8<64, 2>{})
             : go(cache_write8_kernel<0, 2>, Write8<0, 2>{});
}

}  // namespace mla
