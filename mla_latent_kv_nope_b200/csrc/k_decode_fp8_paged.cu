// Split-KV latent decode over a paged 8-bit cache (simple form: CUDA cores).
//
// A page holds 64 rows [512 E4M3 codes || d_r bf16 RoPE keys], all in units of
// the page's scale.  Per sequence b and head i, over the keys of one work range:
//   s_j = softmax_scale * scale_page * (q_cat[b,i] . row_j),  online softmax,
//   o = sum_j p_j scale_page codes_j
// One warp per head; a block stages 32 key rows at a time in shared memory.
#include <cuda_fp8.h>

#include "kernels.h"

namespace mla {

namespace {

constexpr int kHeads = 8;
constexpr int kKeys = 32;
constexpr int kDc = 512;

__global__ void __launch_bounds__(kHeads * 32)
decode8_simt_kernel(const __nv_bfloat16* __restrict__ q_cat, const uint8_t* __restrict__ pool,
                    const float* __restrict__ page_scales, const PageMap pm,
                    const int32_t* __restrict__ seqlens, int B, int H, int d_r, int64_t cap,
                    float scale, int W, float* __restrict__ o_part, float* __restrict__ lse_part,
                    int* __restrict__ status) {
  extern __shared__ float smem[];
  const int R = kDc + d_r, ldr = R + 1, row_bytes = kDc + 2 * d_r;
  float* s_rows = smem;
  float* s_q = s_rows + kKeys * ldr;
  const int w = blockIdx.x, h0 = blockIdx.y * kHeads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, head = h0 + warp;
  pdl_wait();
  int64_t n_units = 0;
  for (int b = 0; b < B; ++b) n_units += units_of(clamp_len(seqlens[b], cap));
  if (n_units == 0) return;
  const int64_t u0 = worker_tile_begin(w, n_units, W), u1 = worker_tile_begin(w + 1, n_units, W);
  if (u0 >= u1) return;
  int64_t prefix = 0;
  for (int b = 0; b < B && prefix < u1; ++b) {
    const int64_t L = clamp_len(seqlens[b], cap), nt = tiles_of(L), r0 = prefix + kSwitchUnits;
    const int64_t lo = max(r0, u0), hi = min(r0 + nt, u1);
    prefix += units_of(L);
    if (nt == 0 || lo >= hi) continue;
    const int64_t key_lo = (lo - r0) * kTileKeys, key_hi = min((hi - r0) * int64_t(kTileKeys), L);
    __syncthreads();
    for (int i = threadIdx.x; i < kHeads * R; i += blockDim.x) {
      const int h = h0 + i / R;
      s_q[i] = h < H ? __bfloat162float(q_cat[(int64_t(b) * H + h) * R + i % R]) : 0.f;
    }
    float m = -INFINITY, l = 0.f, acc[kDc / 32];
#pragma unroll
    for (int k = 0; k < kDc / 32; ++k) acc[k] = 0.f;
    for (int64_t k0 = key_lo; k0 < key_hi; k0 += kKeys) {
      const int nk = int(min(int64_t(kKeys), key_hi - k0));
      const int64_t row0 = pm.row(b, k0);   // 32 keys never cross a page
      const float sc = row0 < 0 ? 0.f : page_scales[row0 / kTileKeys];
      if (row0 < 0 && threadIdx.x == 0) record_status(status, MLA_ERR_BOUNDS);
      __syncthreads();
      for (int i = threadIdx.x; i < nk * R; i += blockDim.x) {
        const int j = i / R, c = i % R;
        float v = 0.f;
        if (row0 >= 0) {
          const uint8_t* row = pool + (row0 + j) * row_bytes;
          if (c < kDc) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(row[c], __NV_E4M3);
            v = __half2float(__half(hr)) * sc;
          } else {
            v = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row + kDc)[c - kDc]) * sc;
          }
        }
        s_rows[j * ldr + c] = v;
      }
      __syncthreads();
      float s = -INFINITY;
      if (lane < nk) {
        const float* q = s_q + warp * R;
        const float* r = s_rows + lane * ldr;
        float a = 0.f;
        for (int c = 0; c < R; ++c) a = fmaf(q[c], r[c], a);
        s = a * scale;
      }
      const float m_new = fmaxf(m, warp_max(s));
      const float p = lane < nk ? expf(s - m_new) : 0.f;
      const float alpha = expf(m - m_new);
      l = l * alpha + warp_sum(p);
      m = m_new;
#pragma unroll
      for (int k = 0; k < kDc / 32; ++k) acc[k] *= alpha;
      for (int j = 0; j < nk; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p, j);
        const float* r = s_rows + j * ldr;
#pragma unroll
        for (int k = 0; k < kDc / 32; ++k) acc[k] = fmaf(pj, r[lane + 32 * k], acc[k]);
      }
    }
    if (head < H) {
      const int slot = b + w;
      const float inv_l = 1.f / l;
      float* o = o_part + int64_t(slot) * kDc * H + int64_t(head) * 4;
#pragma unroll
      for (int k = 0; k < kDc / 32; ++k) {
        const int c = lane + 32 * k;
        o[int64_t(c >> 2) * H * 4 + (c & 3)] = acc[k] * inv_l;
      }
      if (lane == 0) lse_part[int64_t(slot) * H + head] = m + logf(l);
    }
  }
}

}  // namespace

int decode_fp8_paged_splits(int sms, int H) {
  const int groups = (H + kHeads - 1) / kHeads;
  return (2 * sms + groups - 1) / groups;
}

cudaError_t launch_decode_fp8_paged(const __nv_bfloat16* q_cat, const uint8_t* pool,
                                    const float* page_scales, const PageMap& pm,
                                    const int32_t* seqlens, int B, int H, int d_r, int64_t cap,
                                    float scale, int W, float* o_part, float* lse_part,
                                    int* status, uint64_t, cudaStream_t stream) {
  const int R = kDc + d_r;
  const size_t smem = sizeof(float) * (size_t(kKeys) * (R + 1) + size_t(kHeads) * R);
  cudaError_t e = cudaFuncSetAttribute(decode8_simt_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(decode8_simt_kernel, dim3(W, (H + kHeads - 1) / kHeads), dim3(kHeads * 32),
                    smem, stream, q_cat, pool, page_scales, pm, seqlens, B, H, d_r, cap, scale, W,
                    o_part, lse_part, status);
}

}  // namespace mla
