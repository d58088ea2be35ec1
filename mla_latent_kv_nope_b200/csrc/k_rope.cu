// Rotary positions: y = a R(pos) x over the d_r-wide rows of a strided [tokens,
// heads, d_r] view (or the transposed rotation a R(pos)^T, its gradient).
//   y1 = a (x1 cos - x2 sin),  y2 = a (x1 sin + x2 cos)    for each pair (x1, x2)
// A pair is (x[k], x[k + d_r/2]) in the half layout and (x[2k], x[2k+1]) in the
// interleaved one.
//
// Bound by HBM (one read and one write of the rows); small calls by latency.
// A thread moves 8 pairs with 16-byte accesses and issues its loads before the
// cosines and sines are formed, once per (token, pair) of the block, in shared
// memory: with 128 heads that is one sincospif per 128 rotated pairs.  Measured on
// B200: 4096 tokens x 128 heads x 64 bf16 21.3 us (6.3 TB/s, 0.96 of a copy; 25.9
// with one row per thread); 64 x 64 rows 2.1 us, 1023 x 16 fp32 rows 3.3 us.  With one
// head (keys) the angles bound it: 1000 rows 2.0 us, 200,000 rows 23.8 us (55 with the
// table read for every angle, 5.4 us for 1000 rows with 64 tokens a block).
#include "kernels.h"
#include "rope_table.cuh"

namespace mla {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 8;   // pairs per thread
constexpr int kRopeSpread = 592;   // blocks, four to an SM

template <typename T> struct RopeVec;   // 8 values of T as 16-byte words
template <> struct RopeVec<__nv_bfloat16> {
  uint4 v;
  __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct RopeVec<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// Block = `toks` tokens x kBlocks * `heads` heads, one thread per 8 pairs of
// kBlocks rows (toks * heads * (d_r / 16) <= kRopeThreads).  d_r % 16 == 0,
// 16-byte aligned rows.
template <typename T, int kBlocks>
__global__ void __launch_bounds__(kRopeThreads)
rope_vec_kernel(const __grid_constant__ mla_rope_table tab, const T* __restrict__ x, int64_t xt,
                int64_t xh, const int32_t* __restrict__ pos, T* y, int64_t yt, int64_t yh,
                int64_t n_tokens, int H, int toks, int heads, int transpose) {
  __shared__ float2 s_cs[kRopeThreads * kRopePairs];
  const int half = tab.d_r / 2, tpr = tab.d_r / 16;
  const int64_t tok0 = int64_t(blockIdx.x) * toks;
  const int row = threadIdx.x / tpr, g = threadIdx.x % tpr;
  const int tl = row / heads;
  const int64_t tok = tok0 + tl;
  const int head0 = blockIdx.y * kBlocks * heads + row % heads;
  const bool live = tl < toks && tok < n_tokens;
  const bool inter = tab.layout == MLA_ROPE_INTERLEAVED;
  const int o1 = inter ? 16 * g : 8 * g, o2 = inter ? 16 * g + 8 : half + 8 * g;
  // This thread's angles: one pair, every groups-th token.  (Lanes differ in their
  // pair, so the table's read is serialised: once, before the wait.)
  const int groups = kRopeThreads / half, pair = threadIdx.x % half;
  const uint64_t turn = tab.turn[pair];
  pdl_wait();
  RopeVec<T> v1[kBlocks], v2[kBlocks];
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    const int head = head0 + k * heads;
    if (live && head < H) {
      const T* p = x + tok * xt + head * xh;
      v1[k].load(p + o1);
      v2[k].load(p + o2);
    }
  }
  for (int t = threadIdx.x / half; t < toks; t += groups) {
    if (tok0 + t < n_tokens && threadIdx.x < groups * half) {
      float2 cs;
      rope_turn_cos_sin(turn, pos[tok0 + t], tab.amplitude, &cs.x, &cs.y);
      if (transpose) cs.y = -cs.y;
      s_cs[t * half + pair] = cs;
    }
  }
  __syncthreads();
  if (!live) return;
  const float2* cs = s_cs + tl * half + 8 * g;
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    const int head = head0 + k * heads;
    if (head >= H) break;
    float a[8], b[8];
    v1[k].get(a);
    v2[k].get(b);
    if (inter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c0 = cs[i], c1 = cs[4 + i];
        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
        a[2 * i] = a0 * c0.x - a1 * c0.y;
        a[2 * i + 1] = a0 * c0.y + a1 * c0.x;
        b[2 * i] = b0 * c1.x - b1 * c1.y;
        b[2 * i + 1] = b0 * c1.y + b1 * c1.x;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 c = cs[i];
        const float x1 = a[i], x2 = b[i];
        a[i] = x1 * c.x - x2 * c.y;
        b[i] = x1 * c.y + x2 * c.x;
      }
    }
    v1[k].set(a);
    v2[k].set(b);
    T* q = y + tok * yt + head * yh;
    v1[k].store(q + o1);
    v2[k].store(q + o2);
  }
}

// Any even d_r and any strides: one thread per pair.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads)
rope_pair_kernel(const __grid_constant__ mla_rope_table tab, const T* x, int64_t xt, int64_t xh,
                 const int32_t* __restrict__ pos, T* y, int64_t yt, int64_t yh, int64_t n_tokens,
                 int H, int transpose) {
  pdl_wait();
  const int half = tab.d_r / 2;
  const int64_t n = n_tokens * H * half;
  const bool inter = tab.layout == MLA_ROPE_INTERLEAVED;
  for (int64_t i = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * kRopeThreads) {
    const int k = int(i % half);
    const int64_t r = i / half, t = r / H, h = r % H;
    float c, s;
    rope_turn_cos_sin(tab.turn[k], pos[t], tab.amplitude, &c, &s);
    if (transpose) s = -s;
    const int o1 = inter ? 2 * k : k, o2 = inter ? 2 * k + 1 : k + half;
    const T* p = x + t * xt + h * xh;
    T* q = y + t * yt + h * yh;
    const float x1 = Storage<T>::to_f(p[o1]), x2 = Storage<T>::to_f(p[o2]);
    q[o1] = Storage<T>::from_f(x1 * c - x2 * s);
    q[o2] = Storage<T>::from_f(x1 * s + x2 * c);
  }
}

inline bool rows16(const void* p, int64_t a, int64_t b, size_t elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (a * int64_t(elem)) % 16 == 0 &&
         (b * int64_t(elem)) % 16 == 0;
}

}  // namespace

template <typename T>
cudaError_t launch_rope(const mla_rope_table& tab, int64_t n_tokens, int H, const T* x, int64_t xt,
                        int64_t xh, const int32_t* pos, T* y, int64_t yt, int64_t yh,
                        int transpose, cudaStream_t stream) {
  // 16-byte rows take the vector kernel; a width or a stride that is not a
  // multiple of 16 bytes falls to the pair kernel (2-byte accesses).
  if (tab.d_r % 16 == 0 && rows16(x, xt, xh, sizeof(T)) && rows16(y, yt, yh, sizeof(T))) {
    const int rows = kRopeThreads / (tab.d_r / 16);
    const int heads = H < rows ? H : rows;
    // With few heads a block's angles take several rounds of its threads; blocks of
    // fewer tokens, while they all run at once, share them out.
    const int most = rows / heads, once = kRopeThreads / (tab.d_r / 2);
    const int64_t spread = (n_tokens + kRopeSpread - 1) / kRopeSpread;
    const int toks = int(spread >= most || once >= most ? most : spread > once ? spread : once);
    // Two rows a thread where a token has that many heads: twice the loads in
    // flight and half the angles.
    const int blocks = sizeof(T) == 2 && H >= 2 * heads ? 2 : 1;
    const dim3 grid(unsigned((n_tokens + toks - 1) / toks),
                    unsigned((H + blocks * heads - 1) / (blocks * heads)));
    return launch_pdl(blocks == 2 ? rope_vec_kernel<T, 2> : rope_vec_kernel<T, 1>, grid,
                      dim3(kRopeThreads), 0, stream, tab, x, xt, xh, pos, y, yt, yh, n_tokens, H,
                      toks, heads, transpose);
  }
  const int64_t n = n_tokens * H * (tab.d_r / 2);
  const int64_t blocks = (n + kRopeThreads - 1) / kRopeThreads;
  return launch_pdl(rope_pair_kernel<T>, dim3(unsigned(blocks < 8192 ? blocks : 8192)),
                    dim3(kRopeThreads), 0, stream, tab, x, xt, xh, pos, y, yt, yh, n_tokens, H,
                    transpose);
}

template cudaError_t launch_rope<float>(const mla_rope_table&, int64_t, int, const float*, int64_t,
                                        int64_t, const int32_t*, float*, int64_t, int64_t, int,
                                        cudaStream_t);
template cudaError_t launch_rope<__nv_bfloat16>(const mla_rope_table&, int64_t, int,
                                                const __nv_bfloat16*, int64_t, int64_t,
                                                const int32_t*, __nv_bfloat16*, int64_t, int64_t,
                                                int, cudaStream_t);

}  // namespace mla
