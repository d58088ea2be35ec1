// Split-KV latent decode over a paged 8-bit cache for up to 64 heads (sm_100a,
// d_c = 512, d_r = 64 or 0): one CTA per worker, M = 64 products.
//
// The mathematics, the two-term operands and the moving softmax reference are
// those of the CTA-pair kernel (k_decode_fp8_paged.cu).  With at most 64 heads
// half of a pair's rows would be padding and its tile would be staged by two
// CTAs; here every SM takes tiles of its own.  An M = 64 product runs at half
// rate, so a 64-key tile costs as many tensor cycles per SM (36 scores' products
// of 33 cycles, 8 of P.C of 129: 2220) as a pair's 128 keys cost each of its two
// SMs, but half the loads and less power, so a higher clock.
// Measured on B200 (decode alone, graphs of ten): 64 sequences of 512 to 32768
// tokens with 64 heads 176-181 us, against 222 with pairs; 4 x 4096 tokens with 16
// heads 11.9 us, against 14.4.  A tile takes 2490 cycles at 1.8 GHz (memory would
// allow 1750), so the tensor pipe bounds long sequences; a short one is bound by
// its start, about 9 us from the lengths to the first partial.  Tried and not
// faster: a fourth stage in the memory of the staged query (182 us), four more warps
// for the query split and the epilogue (11.8 against 12.1 us, then no difference).
//
// Structure (224 threads):
//   warp 4     TMA producer: per 64-key page 4 boxes of codes [64 keys x 128] and
//              one of RoPE keys [64 x 64 bf16] into a 3-stage ring; and the next
//              sequence's query block, as bf16, while the current one is attended
//   warp 5     QK^T: S = Q C^T, Q hi, lo and RoPE part from tensor memory
//   warp 6     P.C: O += P C, P from the stage's RoPE chunk (free once S is done)
//   warps 0-3  query split, softmax, epilogue
// Tensor memory (an M = 64 tile takes 16 of the 32 lanes of each quadrant; lo =
// lanes 0-15, hi = lanes 16-31):
//   lo lanes: cols [0,64), [64,128) S double buffer; [128,256) Q hi, [256,384) Q
//             lo, [384,416) Q RoPE part
//   hi lanes: cols [0,256) O[:, 0:256]; [256,512) O[:, 256:512]
// A row's keys are shared by two threads of a warp (keys 0-31 and 32-63), so the
// softmax needs no meeting of warps.  Every wait is bounded, as in the pair
// kernel.
#include "decode8.cuh"

namespace mla {

namespace {

using namespace decode8;

constexpr int kStages = 3;
constexpr int kStageBytes = 5 * kChunk;   // 4 chunks of codes, 1 of RoPE keys, then P
constexpr int kPChunk = 4;
constexpr int kSoftmaxWarps = 4;
constexpr int kProducerWarp = 4, kQkWarp = 5, kPvWarp = 6;
constexpr int kThreads = 32 * 7;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColQ = 128;    // lo lanes
constexpr uint32_t kHiLanes = 16u << 16;

constexpr uint32_t kIdescQK = idesc_f16_f32(64, 64, false, false);   // E4M3 is format 0 too
constexpr uint32_t kIdescRope = idesc_bf16_f32(64, 64, false, false);
constexpr uint32_t kIdescPV = idesc_f16_f32(64, 256, false, true);

struct Bars {
  uint64_t full[kStages], empty[kStages];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[kStages];   // by stage: a warp a tile ahead of another cannot speak for it
  uint64_t q_raw, q_raw_free, q_ready, o_free, qk_drain, pv_drain, never;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t kOffStage = 0;
constexpr size_t kOffRaw = size_t(kStages) * kStageBytes;       // 9 chunks [64 rows x 64] bf16
constexpr size_t kOffBars = kOffRaw + 9 * kChunk;
constexpr size_t kOffScratch = kOffBars + (sizeof(Bars) + 15) / 16 * 16;
constexpr size_t kSmemBytes = kOffScratch + 16 * sizeof(int64_t);
static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA");

__device__ __forceinline__ void raise_abort(Bars* bars, int* status) {
  bars->abort_flag = 1;
  record_status(status, MLA_ERR_DEVICE_TIMEOUT);
}

template <int kDr>
__global__ void __launch_bounds__(kThreads, 1)
decode8_64_kernel(const __grid_constant__ CUtensorMap tm_codes,
                  const __grid_constant__ CUtensorMap tm_rope,
                  const __grid_constant__ CUtensorMap tm_query,
                  const __nv_bfloat16* __restrict__ q_cat, const float* __restrict__ page_scales,
                  const PageMap pm, const int32_t* __restrict__ seqlens, int B, int H, int64_t cap,
                  float scale_log2, int W, float* __restrict__ o_part,
                  float* __restrict__ lse_part, int* __restrict__ status, uint64_t inject_wait) {
  constexpr int kQueryChunks = (kDc + kDr) / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  const int w = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // What reads nothing of earlier kernels comes before the wait for them.
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
      mbar_init(&bars->p_full[s], kSoftmaxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->s_free[s], kSoftmaxWarps);
    }
    mbar_init(&bars->q_raw, 1);
    mbar_init(&bars->q_raw_free, kSoftmaxWarps);
    mbar_init(&bars->q_ready, kSoftmaxWarps);
    mbar_init(&bars->o_free, kSoftmaxWarps);
    mbar_init(&bars->qk_drain, 1);
    mbar_init(&bars->pv_drain, 1);
    mbar_init(&bars->never, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 32 * kProducerWarp) {
    tma_prefetch_desc(&tm_codes);
    tma_prefetch_desc(&tm_query);
    if (kDr) tma_prefetch_desc(&tm_rope);
  }
  pdl_wait();
  const int32_t len0 = int(threadIdx.x) < B ? seqlens[threadIdx.x] : 0;
  if (warp == kQkWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  } else if (warp == kProducerWarp) {
    if (lane == 0) prefetch_queries(q_cat, int64_t(B) * H * (kDc + kDr) * 2, w, W);
    prefetch_table(pm, B, w, W);
  }
  tc_fence_before();
  Segments seg;       // (its barriers also make tmem_base and the barriers visible)
  const bool busy = find_segments<kThreads>(
      len0, seqlens, B, cap, w, W, reinterpret_cast<int64_t*>(smem + kOffScratch), &seg);
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  uint32_t n_issued = 0, n_queries = 0;   // tiles and query blocks the producer has asked for
  bool ok = true;

  if (!busy) {
    // No units for this worker.
  } else if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    // The query block of sequence b: rows b H .. b H + 63 of q_cat (rows past the
    // sequence's heads are another's, or zeros past the end: not stored).
    auto load_query = [&](int b) {
      if (n_queries > 0 && !(ok = wait_w(&bars->q_raw_free, (n_queries - 1) & 1, abort_flag)))
        return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_raw, kQueryChunks * kChunk);
        for (int c = 0; c < kQueryChunks; ++c)
          tma_load_2d(&tm_query, &bars->q_raw, smem + kOffRaw + c * kChunk, c * 64, b * H);
      }
      __syncwarp();
      ++n_queries;
      return true;
    };
    uint32_t i = 0;
    bool more = seg.next();
    if (more) load_query(seg.cur);
    while (ok && more) {
      PageWalk walk(pm, nullptr, seg.cur, seg.lo, seg.hi);
      const int64_t lo = seg.lo, hi = seg.hi;
      for (int64_t t = lo; t < hi; ++t, ++i) {
        const int st = i % kStages;
        int64_t r;
        float unused;
        walk.at(t, &r, &unused);
        if (i >= kStages && !(ok = wait_w(&bars->empty[st], (i / kStages - 1) & 1, abort_flag)))
          break;
        if (lane == 0) {
          if (r < 0) {   // reads as zeros: past the end of the map
            record_status(status, MLA_ERR_BOUNDS);
            r = pm.total_rows(B);
          }
          uint8_t* dst = smem + kOffStage + st * kStageBytes;
          mbar_arrive_expect_tx(&bars->full[st], (kDr ? 5 : 4) * kChunk);
          for (int c = 0; c < 4; ++c)
            tma_load_2d(&tm_codes, &bars->full[st], dst + c * kChunk, c * 128, int32_t(r));
          if (kDr)
            tma_load_2d(&tm_rope, &bars->full[st], dst + kPChunk * kChunk, kDc / 2, int32_t(r));
        }
        __syncwarp();
        n_issued = i + 1;
      }
      if (!ok) break;
      more = seg.next();
      if (more) load_query(seg.cur);
    }
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ QK^T
    uint32_t i = 0, n_seg = 0;
    const uint64_t kd = smem_desc_sw128(smem_u32(smem + kOffStage), 16, 1024);
    // Test hook: a wait on a barrier nothing arrives on, so the give-up path runs.
    if (inject_wait) ok = wait_w(&bars->never, 0, abort_flag, inject_wait);
    for (; ok && seg.next(); ++n_seg) {
      if (!(ok = wait_w(&bars->q_ready, n_seg & 1, abort_flag))) break;
      for (int64_t t = seg.lo; t < seg.hi; ++t, ++i) {
        const int st = i % kStages, sb = i & 1;
        if (!(ok = wait_w(&bars->full[st], (i / kStages) & 1, abort_flag)) ||
            (i >= 2 && !(ok = wait_w(&bars->s_free[sb], ((i >> 1) - 1) & 1, abort_flag))))
          break;
        tc_fence_after();
        const uint32_t d = tmem + kColS + uint32_t(sb) * 64u;
        const uint64_t b0 = kd + uint64_t((uint32_t(st) * kStageBytes) >> 4);
#pragma unroll 1
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int term = 0; term < 2; ++term)
              mma_f8_ts_w(d, tmem + kColQ + uint32_t(term) * 128u + uint32_t(c * 4 + k) * 8u,
                          b0 + uint64_t((c * kChunk + k * 32) >> 4), kIdescQK, (c | k | term) != 0);
        if (kDr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ts_w(d, tmem + kColQ + 256u + uint32_t(k) * 8u,
                          b0 + uint64_t((kPChunk * kChunk + k * 32) >> 4), kIdescRope, true);
        }
        mma_commit_w(&bars->s_full[sb]);
      }
    }
    mma_commit_w(&bars->qk_drain);
    volatile int no_abort = 0;
    wait_w(&bars->qk_drain, 0, &no_abort);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ P.C
    uint32_t i = 0, n_seg = 0;
    const uint64_t pd = smem_desc_sw128(smem_u32(smem + kOffStage + kPChunk * kChunk), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_u32(smem + kOffStage), kChunk, 1024);
    for (; ok && seg.next(); ++n_seg) {
      for (int64_t t = seg.lo; t < seg.hi; ++t, ++i) {
        const int st = i % kStages;
        // The previous sequence's epilogue has read O before it is overwritten.
        if (t == seg.lo && n_seg > 0 && !(ok = wait_w(&bars->o_free, (n_seg - 1) & 1, abort_flag)))
          break;
        if (!(ok = wait_w(&bars->p_full[st], (i / kStages) & 1, abort_flag))) break;
        tc_fence_after();
        const uint64_t off = uint64_t((uint32_t(st) * kStageBytes) >> 4);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_f8_ss_w(tmem + kHiLanes + uint32_t(h) * 256u,
                          pd + off + uint64_t((term * 64 + k * 32) >> 4),
                          vd + off + uint64_t((2 * h * kChunk + k * 32 * 128) >> 4),
                          term ? kIdescPV | kE5m2A : kIdescPV,
                          !(t == seg.lo && k == 0 && term == 0));
        mma_commit_w(&bars->empty[st]);
      }
    }
    mma_commit_w(&bars->pv_drain);
    volatile int no_abort = 0;
    wait_w(&bars->pv_drain, 0, &no_abort);
  } else {
    // ------------------------------------------------------------ softmax
    const int tid = threadIdx.x;             // 0..127
    const int half = lane >> 4;              // keys 0-31 or 32-63 of a tile
    const int row = 16 * warp + (lane & 15); // head row
    const uint32_t lo_base = tmem + (uint32_t(32 * warp) << 16);
    const uint32_t hi_base = lo_base + kHiLanes;
    uint32_t i = 0, n_seg = 0;
    auto arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };

    // Splits the staged query block into E4M3 terms in tensor memory.  A thread
    // takes every second 16 values of its row (the two threads of a row the
    // others'), reads them once for the row's largest value and once more to
    // split them; a 16x32bx2 store puts the pair's 4 columns side by side.
    // Returns the row's factor 2^k.
    float row_factor = 0.f;
    auto write_query = [&] {
      if (!(ok = wait_w(&bars->q_raw, n_seg & 1, abort_flag))) return false;
      const uint8_t* raw = smem + kOffRaw + row * 128;
      // 16-byte unit u of the row (8 values), in chunk u / 8.
      auto unit = [&](int u) {
        return *reinterpret_cast<const uint4*>(raw + (u / 8) * kChunk + (((u % 8) ^ (row & 7)) * 16));
      };
      uint32_t top = 0;
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const uint4 a = unit(4 * j + 2 * half), b = unit(4 * j + 2 * half + 1);
        // bf16 bits order like their magnitudes.
        top = max_magnitude2(max_magnitude2(max_magnitude2(max_magnitude2(top, a.x), a.y), a.z), a.w);
        top = max_magnitude2(max_magnitude2(max_magnitude2(max_magnitude2(top, b.x), b.y), b.z), b.w);
      }
      top = larger_half(top);
      if (kDr) {
        uint32_t rope = 0;
#pragma unroll
        for (int j = 0; j < kDr / 16; ++j) {
          const uint4 a = unit(64 + 2 * j + half);
          rope = max_magnitude2(max_magnitude2(max_magnitude2(max_magnitude2(rope, a.x), a.y), a.z), a.w);
        }
        top = max(top, rope_magnitude(larger_half(rope)));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const int k = query_exponent(top);
      const __nv_bfloat162 inv = __float2bfloat162_rn(exp2i(-k));
      row_factor = exp2i(k);
#pragma unroll 4
      for (int j = 0; j < 16; ++j) {
        const uint4 a = unit(4 * j + 2 * half), b = unit(4 * j + 2 * half + 1);
        const uint32_t wd[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) split_query(wd[x], inv, &hi[x], &lo[x]);
        tmem_st16x2_4<4>(lo_base + kColQ + uint32_t(8 * j),
                         make_uint4(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16),
                                    hi[4] | (hi[5] << 16), hi[6] | (hi[7] << 16)));
        tmem_st16x2_4<4>(lo_base + kColQ + 128u + uint32_t(8 * j),
                         make_uint4(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16),
                                    lo[4] | (lo[5] << 16), lo[6] | (lo[7] << 16)));
      }
      if (kDr) {
#pragma unroll 1
        for (int j = 0; j < kDr / 16; ++j) {
          uint4 a = unit(64 + 2 * j + half);
          a.x = scale_bf16x2(a.x, inv), a.y = scale_bf16x2(a.y, inv);
          a.z = scale_bf16x2(a.z, inv), a.w = scale_bf16x2(a.w, inv);
          tmem_st16x2_4<4>(lo_base + kColQ + 256u + uint32_t(8 * j), a);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      arrive(&bars->q_raw_free);
      if (lane == 0) mbar_arrive(&bars->q_ready);
      return true;
    };

    bool more = seg.next();
    if (more) more = write_query();
    while (more) {
      const int b = seg.cur;
      const int64_t lo = seg.lo, hi = seg.hi, L = seg.L;
      const float row_scale = row_factor * scale_log2;
      PageWalk walk(pm, page_scales, b, lo, hi);
      float ref = 0.f, top = 0.f, l_sum = 0.f;         // set by the first tile
      for (int64_t t = lo; t < hi; ++t, ++i) {
        const int st = i % kStages, sb = i & 1;
        int64_t unused;
        float sc;                // the page's scale
        walk.at(t, &unused, &sc);
        if (!(ok = wait_w(&bars->s_full[sb], (i >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        uint32_t x[32];          // keys 32 half .. of the page
        tmem_ld16x2_32<32>(lo_base + kColS + uint32_t(sb) * 64u, x);
        tmem_wait_ld();
        tc_fence_before();
        arrive(&bars->s_free[sb]);

        uint8_t* stage = smem + kOffStage + st * kStageBytes;
        const int valid = int(min(L - t * kTileKeys, int64_t(kTileKeys)));
        if (valid < kTileKeys) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 * half + j >= valid) x[j] = 0xFF800000u;   // -inf
          // Rows past the sequence's end may hold anything, NaN codes among it:
          // their weight is 0, so they are zeroed in the staged page.
          for (int u = tid; u < (kTileKeys - valid) * 32; u += 32 * kSoftmaxWarps)
            *reinterpret_cast<uint4*>(stage + (u & 3) * kChunk + (valid + u / 32) * 128 +
                                      ((u / 4) % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(x[j]));
        const float f = score_factor(row_scale, sc), lsc = log2f(sc);
        // log2 of the largest p * scale of the row's 64 keys.
        float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * f + lsc;
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
        float alpha = 1.f;
        if (t == lo) {
          top = mt;
          ref = mt + kLeadFirst;
        } else {
          top = fmaxf(top, mt);
          const float next = next_reference(ref, mt, top);
          if (next != ref) {
            alpha = ex2_approx(ref - next);
            ref = next;
            l_sum *= alpha;
          }
        }
        uint32_t hi8[8], lo8[8];
        const float sum = split_probabilities(x, f, lsc + kPScale - ref, hi8, lo8);
        l_sum = fmaf(sum, 1.f / sc, l_sum);
        // P into the stage's RoPE chunk, rows of [64 hi, 64 lo].
        uint8_t* prow = stage + kPChunk * kChunk + row * 128;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int un = half * 2 + u;
          *reinterpret_cast<uint4*>(prow + (un ^ (row & 7)) * 16) =
              make_uint4(hi8[4 * u], hi8[4 * u + 1], hi8[4 * u + 2], hi8[4 * u + 3]);
          *reinterpret_cast<uint4*>(prow + ((un + 4) ^ (row & 7)) * 16) =
              make_uint4(lo8[4 * u], lo8[4 * u + 1], lo8[4 * u + 2], lo8[4 * u + 3]);
        }
        if (t != lo && __any_sync(0xffffffffu, alpha != 1.f)) {
          const uint32_t prev = i - 1;                 // O holds P.C(i - 1)
          if (!(ok = wait_w(&bars->empty[prev % kStages], (prev / kStages) & 1, abort_flag))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            uint32_t r[32];
            tmem_ld16x2_32<256>(hi_base + uint32_t(c), r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16x2_32<256>(hi_base + uint32_t(c), r);
          }
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(&bars->p_full[st]);
      }
      if (!ok) break;
      // Every QK^T of this sequence has been read back: load the next query.
      more = seg.next();
      ++n_seg;
      if (more && !write_query()) break;
      // Epilogue: normalised partial output and log-sum-exp.
      const uint32_t last = i - 1;
      if (!(ok = wait_w(&bars->empty[last % kStages], (last / kStages) & 1, abort_flag))) break;
      tc_fence_after();
      const float l_row = l_sum + __shfl_xor_sync(0xffffffffu, l_sum, 16);
      const float inv = 1.f / l_row;
      const int slot = b + w;
      // Partials are o_part[slot][d_c / 4][H][4]: lanes 0-15 store 16 consecutive
      // heads of one 4-column group, lanes 16-31 the same heads 64 groups on; kept
      // in L2 for the combine that reads them next.
      float* dst = o_part + ((int64_t(slot) * (kDc / 4) + half * 64) * H + row) * 4;
      const uint64_t keep = l2_policy_evict_last();
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t r[32];
        tmem_ld16x2_32<256>(hi_base + uint32_t(c), r);
        tmem_wait_ld();
        if (row < H) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            st_global_f4_hint(dst + int64_t(c / 4 + e) * H * 4,
                              make_float4(__uint_as_float(r[4 * e]) * inv,
                                          __uint_as_float(r[4 * e + 1]) * inv,
                                          __uint_as_float(r[4 * e + 2]) * inv,
                                          __uint_as_float(r[4 * e + 3]) * inv),
                              keep);
        }
      }
      if (half == 0 && row < H)
        lse_part[int64_t(slot) * H + row] = (log2f(l_row) + ref - kPScale) * 0.69314718055994531f;
      tc_fence_before();
      arrive(&bars->o_free);
    }
  }
  if (!ok && lane == 0) raise_abort(bars, status);

  // Every role has stopped.  Each load the producer issued lands before the
  // shared memory is released (after a give-up some were never waited for).
  __syncwarp();
  if (warp == kProducerWarp && lane == 0) {
    volatile int no_abort = 0;
    for (uint32_t k = (n_issued > kStages ? n_issued - kStages : 0); k < n_issued; ++k)
      mbar_wait(&bars->full[k % kStages], (k / kStages) & 1, &no_abort, kWaitLimitCycles / 100);
    if (n_queries) mbar_wait(&bars->q_raw, (n_queries - 1) & 1, &no_abort, kWaitLimitCycles / 100);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int kDr, typename... Args>
cudaError_t launch_t(dim3 grid, cudaStream_t stream, Args... args) {
  static bool attr_done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode8_64_kernel<kDr>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(kSmemBytes));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl(decode8_64_kernel<kDr>, grid, dim3(kThreads), kSmemBytes, stream, args...);
}

}  // namespace

cudaError_t launch_decode_fp8_paged64(const CUtensorMap& tm_codes, const CUtensorMap& tm_rope,
                                      const CUtensorMap& tm_query, const __nv_bfloat16* q_cat, const float* page_scales,
                                      const PageMap& pm, const int32_t* seqlens, int B, int H,
                                      int d_r, int64_t cap, float scale_log2, int W, float* o_part,
                                      float* lse_part, int* status, uint64_t inject_wait,
                                      cudaStream_t stream) {
  const dim3 grid(W);
  if (d_r)
    return launch_t<64>(grid, stream, tm_codes, tm_rope, tm_query, q_cat, page_scales, pm, seqlens, B, H,
                        cap, scale_log2, W, o_part, lse_part, status, inject_wait);
  return launch_t<0>(grid, stream, tm_codes, tm_rope, tm_query, q_cat, page_scales, pm, seqlens, B, H, cap,
                     scale_log2, W, o_part, lse_part, status, inject_wait);
}

}  // namespace mla
