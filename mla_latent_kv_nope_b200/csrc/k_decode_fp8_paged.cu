// Split-KV latent decode over a paged 8-bit cache for sm_100a (d_c = 512, d_r =
// 64 or 0).
//
// A page holds 64 rows [512 E4M3 codes || d_r bf16 RoPE keys], all in units of
// the page's power-of-two scale.  Per sequence b and head i, over the keys of
// one work range:
//   s_j = softmax_scale * scale_page * (q_cat[b,i] . row_j),  softmax over j,
//   o = sum_j p_j scale_page codes_j
//
// 8-bit products without widening.  The codes go to the tensor cores as they
// lie in the cache (kind::f8f6f4, twice the 16-bit rate); what is not 8 bits is
// split into two terms, x = hi + lo:
//   * a query row times a power of two (largest latent value in (224, 448], smaller
//     where the rotary part is 2^40 times larger) into E4M3 + E4M3: a bf16 value
//     has 8 significant bits and each term holds 4, so hi + lo is exact for values
//     within 2^10 of the largest, and off by at most 2^-18 of it below;
//   * a probability into E4M3 + E5M2: hi is off by at most 2^-4 of p, lo by 2^-3
//     of that, 2^-7 of p together, or 2^-17 where lo is below E5M2's normal numbers
//     (1.4e-3 of the output in a simulation of scores with a deviation of 0.3 to
//     3.5, as for bf16 probabilities).
// So both products cost as many tensor cycles as 16-bit ones, but the cache
// is read, staged and fed at one byte per value and no thread touches it.  The
// RoPE part is a bf16 product into the same accumulator.
// The page scale folds into the probability (p_j scale_page enters the second
// product), so it costs one multiply per key and head group.
//
// Range of the probabilities.  With one reference (a running maximum) keys far
// below the largest of the whole sequence would vanish in 8 bits, and
// thousands of those can carry most of the weight (one early key that
// outweighs all others).  The reference r therefore follows the tile: it moves
// when a tile's maximum leaves [r - kFall, r + kRise] (log2), up or down, with O
// and l rescaled by 2^(r_old - r_new) in fp32; it stays within 2^60 of the
// largest so far, below which nothing is left to add.  A move costs a wait for
// the last product, so the window is as wide as the two formats allow: E5M2 lo
// holds what E4M3 hi loses down to 2^-16, so a tile whose maximum lies 2^13
// below the reference still keeps three bits of keys 2^7 below that; 2^-17 is
// then 2^-10.7 of its largest, and keys 2^11 below that are lost from O (the sum l,
// in fp32, counts them).  With E4M3 for lo the window was 2^7 wide and two tiles in three moved some row of 128
// (scores with a deviation of 1.7); now one in forty does.
//
// Structure: a cluster of two CTAs (128 heads, 64 each) shares every product
// with cta_group::2, M = 128.  One CTA alone could not: 128 heads x 512 output
// columns of fp32 fill its tensor memory, and M = 64 products run at half rate.
// With the pair each CTA holds its 64 heads' O in 256 columns (an M = 128 pair
// accumulator keeps columns [0, N/2) in lanes 0-63 and [N/2, N) in lanes
// 64-127).  Per tile of two pages (128 keys):
//   S [64 heads each, 128 keys] = Q . K^T: CTA r supplies page r's rows
//   O [64 heads each, 512] += P . C:     CTA r supplies columns [128 r, +128) and
//                                        [256 + 128 r, +128) of both pages
// A CTA thus stages its own page whole (K: codes and RoPE keys, 40 KB, 2
// stages) and half the columns of both pages again (V: 16 KB per page, 3
// stages; out of L2), because the operands of a pair product must lie at the
// same offsets in both CTAs.
//   warps 0-7  softmax: thread = (head row, page, half of the page's keys);
//              query split, epilogue
//   warp 8     K loads (TMA);  warp 10  V loads
//   warp 9     QK^T products (leader); in the other CTA it tells the leader that
//              a K stage has landed
//   warp 11    P.C products (leader); the same for V.  Two issuing warps: a
//              product's issue blocks while the tensor pipe is busy, and the waits
//              before one are hidden behind the other's products
// The softmax loop is kept short: with 64 keys a thread, unrolled, its code
// overran the instruction cache and a tile took 5300 cycles, most of them
// waiting for instructions.  Arrivals on the other CTA's barriers have CTA scope
// (see mbar_arrive_cluster): at cluster scope a tile took 900 cycles more.
//
// Measured on B200, 32 x 8192 tokens, 128 heads (decode alone, graphs of ten): 64.5
// us, 79 us when repeated without a pause (the clock drops: the products draw
// the power).  A tile takes 2565 cycles; its products alone 2272 (36 of 33.4
// cycles and 16 of 67, by a microbenchmark), its shared-memory traffic 2600 at 128
// bytes a cycle.  About 14,000 cycles go by before the first scores (setup, the
// query block's copy and split), 4,000 in an epilogue.  Memory would allow 26 us,
// the bf16 kernel over a bf16 cache takes 92, the fp16-widening 8-bit kernel 128.
// Tried and not faster: Q hi from tensor memory (less shared-memory traffic,
// 68.6 us), softmax groups that take tiles in turn (71.0), other orders of the
// products' terms.
// Every wait is bounded (about 2 s of SM cycles); on give-up a CTA raises the
// abort flag of both, records MLA_ERR_DEVICE_TIMEOUT, drains its own loads and
// products and exits.
#include "decode8.cuh"

namespace mla {

namespace {

using namespace decode8;

constexpr int kKStages = 2, kVStages = 3;   // V, and the pages' P tiles
constexpr int kKBytes = 5 * kChunk;       // 4 chunks of codes, 1 of RoPE keys
constexpr int kVBytes = 2 * kChunk;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
constexpr int kKWarp = kSoftmaxWarps, kQkWarp = kKWarp + 1, kVWarp = kKWarp + 2,
              kPvWarp = kKWarp + 3;
constexpr int kThreads = kSoftmaxThreads + 4 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 256;    // O: 2 x 128 columns, S: 2 x 64

constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128, false, false);   // E4M3 is format 0 too
constexpr uint32_t kIdescRope = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescPV = idesc_f16_f32(128, 256, false, true);

struct Bars {
  uint64_t kfull[kKStages];   // leader's: both CTAs' stages have landed
  uint64_t vfull[kVStages], vempty[kVStages];
  uint64_t s_full[2], s_free[2];
  uint64_t p_full[2], pv_done[2];
  uint64_t q_raw, q_ready, o_free, qk_drain, pv_drain, never;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t kOffQ = 0;                                  // 4 hi, 4 lo, 1 RoPE chunk
constexpr size_t kOffP = kOffQ + 9 * kChunk;                 // rows of [64 hi, 64 lo]
constexpr size_t kOffK = kOffP + size_t(kVStages) * kChunk;
constexpr size_t kOffV = kOffK + size_t(kKStages) * kKBytes;
constexpr size_t kOffBars = kOffV + size_t(kVStages) * kVBytes;
constexpr size_t kOffMax = kOffBars + (sizeof(Bars) + 15) / 16 * 16;   // [2][4][64] floats
constexpr size_t kOffRowScale = kOffMax + 2 * 4 * 64 * sizeof(float);  // [2][64] floats
constexpr size_t kSmemBytes = kOffRowScale + 2 * 64 * sizeof(float);
static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA");

__device__ __forceinline__ void raise_abort(Bars* bars, int* status) {
  for (uint32_t r = 0; r < 2; ++r) st_cluster_u32(cluster_map(&bars->abort_flag, r), 1);
  record_status(status, MLA_ERR_DEVICE_TIMEOUT);
}

template <int kDr>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
decode8_kernel(const __grid_constant__ CUtensorMap tm_codes,
               const __grid_constant__ CUtensorMap tm_rope,
               const __grid_constant__ CUtensorMap tm_query,
               const float* __restrict__ page_scales, const PageMap pm,
               const __nv_bfloat16* __restrict__ q_cat, const int32_t* __restrict__ seqlens, int B,
               int H, int64_t cap, float scale_log2, int W, float* __restrict__ o_part,
               float* __restrict__ lse_part, int* __restrict__ status, uint64_t inject_wait) {
  constexpr int R = kDc + kDr;
  // The swizzled operands need 1024-byte alignment; the kernel has no other
  // shared memory, so the array starts on it.
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);
  const uint32_t rank = cluster_rank();
  const int g = blockIdx.x, w = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // What reads nothing of earlier kernels comes before the wait for them, the
  // meeting with the other CTA too (after it, it would wait for the loads below).
  if (threadIdx.x == 0) {
    // The leader's also wait for the other CTA's word that its stage has landed.
    const uint32_t n_full = rank == 0 ? 2 : 1;
    for (int s = 0; s < kKStages; ++s) mbar_init(&bars->kfull[s], n_full);
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bars->vfull[s], n_full);
      mbar_init(&bars->vempty[s], 1);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&bars->s_full[s], 1), mbar_init(&bars->s_free[s], 2 * kSoftmaxWarps);
    mbar_init(&bars->q_raw, 1);
    mbar_init(&bars->q_ready, 2 * kSoftmaxWarps);   // the softmax warps of both CTAs
    mbar_init(&bars->o_free, 2 * kSoftmaxWarps);
    for (int s = 0; s < 2; ++s)
      mbar_init(&bars->p_full[s], 2 * kSoftmaxWarps), mbar_init(&bars->pv_done[s], 1);
    mbar_init(&bars->qk_drain, 1);
    mbar_init(&bars->pv_drain, 1);
    mbar_init(&bars->never, 1);
    bars->abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 32 * kKWarp) {
    tma_prefetch_desc(&tm_codes);
    tma_prefetch_desc(&tm_query);
    if (kDr) tma_prefetch_desc(&tm_rope);
  }
  cluster_sync();
  pdl_wait();
  const int32_t len0 = int(threadIdx.x) < B ? seqlens[threadIdx.x] : 0;
  if (warp == kQkWarp) {
    tmem_alloc_pair(&bars->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  } else if (warp == kVWarp) {
    const int64_t cta = int64_t(blockIdx.y) * gridDim.x + blockIdx.x,
                  n_cta = int64_t(gridDim.x) * gridDim.y;
    if (lane == 0) prefetch_queries(q_cat, int64_t(B) * H * R * 2, cta, n_cta);
    prefetch_table(pm, B, cta, n_cta);
  }
  tc_fence_before();
  Segments seg;       // (its barriers also make tmem_base visible)
  const bool busy = find_segments<kThreads>(len0, seqlens, B, cap, w, W,
                                            reinterpret_cast<int64_t*>(smem), &seg);
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  uint32_t n_issued = 0;     // K or V stages that this producer warp has loaded into
  bool ok = true;

  if (!busy) {
    // No units: the same in both CTAs of the pair.
  } else if (warp == kKWarp) {
    // ------------------------------------------------------------ K and scales
    uint32_t i = 0;
    while (ok && seg.next()) {
      const int64_t lo = seg.lo, hi = seg.hi;
      PageWalk walk(pm, nullptr, seg.cur, lo, hi);
      for (int64_t t = lo; t < hi; t += 2, ++i) {
        const int st = i & 1;
        const bool two = t + 1 < hi;
        int64_t r = -1;
        float unused;
        if (rank == 0 || two) walk.at(t + rank, &r, &unused);
        if (i >= 2 && !(ok = wait_w(&bars->s_full[st], ((i >> 1) - 1) & 1, abort_flag))) break;
        if (lane == 0) {
          if (rank == 0 || two) {
            if (r < 0) {   // reads as zeros: past the end of the map
              record_status(status, MLA_ERR_BOUNDS);
              r = pm.total_rows(B);
            }
            uint8_t* dst = smem + kOffK + st * kKBytes;
            mbar_arrive_expect_tx(&bars->kfull[st], (kDr ? 5 : 4) * kChunk);
            for (int c = 0; c < 4; ++c)
              tma_load_2d(&tm_codes, &bars->kfull[st], dst + c * kChunk, c * 128, int32_t(r));
            if (kDr) tma_load_2d(&tm_rope, &bars->kfull[st], dst + 4 * kChunk, kDc / 2, int32_t(r));
          } else {
            mbar_arrive(&bars->kfull[st]);   // no second page: its scores are masked
          }
        }
        __syncwarp();
        n_issued = i + 1;
      }
    }
  } else if (warp == kVWarp) {
    // ------------------------------------------------------------ V
    uint32_t v = 0;
    while (ok && seg.next()) {
      PageWalk walk(pm, nullptr, seg.cur, seg.lo, seg.hi);
      for (int64_t t = seg.lo; t < seg.hi; ++t, ++v) {
        const int vs = v % kVStages;
        int64_t r;
        float unused;
        walk.at(t, &r, &unused);
        if (v >= kVStages &&
            !(ok = wait_w(&bars->vempty[vs], (v / kVStages - 1) & 1, abort_flag)))
          break;
        if (lane == 0) {
          if (r < 0) r = pm.total_rows(B);
          uint8_t* dst = smem + kOffV + vs * kVBytes;
          mbar_arrive_expect_tx(&bars->vfull[vs], kVBytes);
          for (int h = 0; h < 2; ++h)
            tma_load_2d(&tm_codes, &bars->vfull[vs], dst + h * kChunk, (2 * h + int(rank)) * 128,
                        int32_t(r));
        }
        __syncwarp();
        n_issued = v + 1;
      }
    }
  } else if (warp == kQkWarp && rank == 0) {
    // ------------------------------------------------------------ QK^T (leader)
    uint32_t i = 0, n_seg = 0;
    const uint64_t qd = smem_desc_sw128(smem_u32(smem + kOffQ), 16, 1024);
    const uint64_t kd = smem_desc_sw128(smem_u32(smem + kOffK), 16, 1024);
    // Test hook: a wait on a barrier nothing arrives on, so the give-up path runs.
    if (inject_wait) ok = wait_w(&bars->never, 0, abort_flag, inject_wait);
    for (; ok && seg.next(); ++n_seg) {
      if (!(ok = wait_w(&bars->q_ready, n_seg & 1, abort_flag))) break;
      for (int64_t t = seg.lo; t < seg.hi; t += 2, ++i) {
        const int st = i & 1;
        const uint32_t ph = (i >> 1) & 1;
        if (!(ok = wait_w(&bars->kfull[st], ph, abort_flag)) ||
            (i >= 2 && !(ok = wait_w(&bars->s_free[st], ph ^ 1, abort_flag))))
          break;
        tc_fence_after();
        const uint32_t d = tmem + kColS + uint32_t(st) * 64u;
        const uint64_t b0 = kd + uint64_t((uint32_t(st) * kKBytes) >> 4);
#pragma unroll 1
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int term = 0; term < 2; ++term)
              mma_f8_ss_pair_w(d, qd + uint64_t(((term * 4 + c) * kChunk + k * 32) >> 4),
                               b0 + uint64_t((c * kChunk + k * 32) >> 4), kIdescQK,
                               (c | k | term) != 0);
        if (kDr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ss_pair_w(d, qd + uint64_t((8 * kChunk + k * 32) >> 4),
                               b0 + uint64_t((4 * kChunk + k * 32) >> 4), kIdescRope, true);
        }
        mma_commit_pair_w(&bars->s_full[st]);
      }
    }
    mma_commit_pair_w(&bars->qk_drain);
    volatile int no_abort = 0;
    wait_w(&bars->qk_drain, 0, &no_abort);
  } else if (warp == kPvWarp && rank == 0) {
    // ------------------------------------------------------------ P.C (leader)
    // A second issuing warp: a product's issue blocks while the tensor pipe is
    // busy, and the waits before one product are hidden behind the other's.
    uint32_t i = 0, v = 0, n_seg = 0;
    const uint64_t pd = smem_desc_sw128(smem_u32(smem + kOffP), 16, 1024);
    const uint64_t vd = smem_desc_sw128(smem_u32(smem + kOffV), kChunk, 1024);
    for (; ok && seg.next(); ++n_seg) {
      for (int64_t t = seg.lo; t < seg.hi; t += 2, ++i) {
        // The previous sequence's epilogue has read O before it is overwritten.
        if (t == seg.lo && n_seg > 0 && !(ok = wait_w(&bars->o_free, (n_seg - 1) & 1, abort_flag)))
          break;
        if (!(ok = wait_w(&bars->p_full[i & 1], (i >> 1) & 1, abort_flag))) break;
#pragma unroll 1
        for (int p = 0; p < 2 && t + p < seg.hi; ++p, ++v) {
          const int vs = v % kVStages;
          if (!(ok = wait_w(&bars->vfull[vs], (v / kVStages) & 1, abort_flag))) break;
          tc_fence_after();
          const uint64_t a0 = pd + uint64_t((uint32_t(vs) * kChunk) >> 4);
          const uint64_t b0 = vd + uint64_t((uint32_t(vs) * kVBytes) >> 4);
          const bool fresh = t == seg.lo && p == 0;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int term = 0; term < 2; ++term)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                mma_f8_ss_pair_w(tmem + kColO + uint32_t(h) * 128u,
                                 a0 + uint64_t((term * 64 + k * 32) >> 4),
                                 b0 + uint64_t((h * kChunk + k * 32 * 128) >> 4),
                                 term ? kIdescPV | kE5m2A : kIdescPV,
                                 !(fresh && k == 0 && term == 0));
          mma_commit_pair_w(&bars->vempty[vs]);
        }
        if (!ok) break;
        mma_commit_pair_w(&bars->pv_done[i & 1]);
      }
    }
    mma_commit_pair_w(&bars->pv_drain);
    volatile int no_abort = 0;
    wait_w(&bars->pv_drain, 0, &no_abort);
  } else if (warp == kQkWarp || warp == kPvWarp) {
    // ------------------------------------------------- landed loads, to the leader
    uint32_t n = 0;
    const bool k_side = warp == kQkWarp;
    while (ok && seg.next()) {
      for (int64_t t = seg.lo; t < seg.hi; t += k_side ? 2 : 1, ++n) {
        uint64_t* full = k_side ? &bars->kfull[n & 1] : &bars->vfull[n % kVStages];
        const uint32_t ph = (k_side ? n >> 1 : n / kVStages) & 1;
        if (!(ok = wait_w(full, ph, abort_flag))) break;
        if (lane == 0) mbar_arrive_cluster(cluster_map(full, 0));
        __syncwarp();
      }
    }
    // The leader's last arrival on this CTA's barriers.
    volatile int no_abort = 0;
    wait_w(k_side ? &bars->qk_drain : &bars->pv_drain, 0, &no_abort);
  } else {
    // ------------------------------------------------------------ softmax
    const int tid = threadIdx.x;             // 0..255
    const int quad = warp & 3, part = warp >> 2;   // tensor-memory lanes; which half of the columns
    const int row = (32 * quad + lane) & 63, pg = quad >> 1;   // head row; page of the pair
    const int head = g * kHeadsPerCta + row;
    const uint32_t lanes = tmem + (uint32_t(32 * quad) << 16);
    float* s_max = reinterpret_cast<float*>(smem + kOffMax);
    float* s_row = reinterpret_cast<float*>(smem + kOffRowScale);
    const uint32_t a_q = cluster_map(&bars->q_ready, 0), a_p0 = cluster_map(&bars->p_full[0], 0),
                   a_p1 = cluster_map(&bars->p_full[1], 0),
                   a_o = cluster_map(&bars->o_free, 0), a_s0 = cluster_map(&bars->s_free[0], 0),
                   a_s1 = cluster_map(&bars->s_free[1], 0);
    uint32_t i = 0, v = 0;
    auto arrive = [&](uint32_t addr) {
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(addr);
    };
    // The softmax warps meet.  This wait has no limit of its own, so a warp that
    // has given up does not leave: it walks on without waiting for anything
    // else, and every warp comes to every meeting.
    auto meet_all = [&] {
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
    };
    // The four warps that share rows (both pages, both parts of 32 rows).
    auto meet = [&] {
      asm volatile("bar.sync %0, %1;" ::"r"(2 + (warp & 1)), "n"(kSoftmaxThreads / 2) : "memory");
    };
    auto await = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = wait_w(bar, parity, abort_flag);
      if (!ok && lane == 0) raise_abort(bars, status);
    };

    // The query block of sequence b (64 rows of q_cat; rows past the sequence's
    // heads are another's, or zeros past the end: not stored) is copied as bf16
    // into the shared memory that its E4M3 terms will take, and split in place: a
    // warp takes 8 rows, two at a time, and has read a row before it writes it.
    // The rows' factors alternate between two buffers: a warp may get here before
    // another has read the last sequence's.
    uint32_t n_query = 0, n_copied = 0;   // query blocks split; copied (by thread 0)
    auto copy_query = [&](int b) {
      fence_proxy_async_smem();   // after what threads have read and written there
      mbar_arrive_expect_tx(&bars->q_raw, (R / 64) * kChunk);
#pragma unroll 1
      for (int c = 0; c < R / 64; ++c)
        tma_load_2d(&tm_query, &bars->q_raw, smem + kOffQ + c * kChunk, c * 64,
                    b * H + g * kHeadsPerCta);
      ++n_copied;
    };
    auto write_query = [&] {
      float* factor = s_row + (n_query & 1) * 64;
      await(&bars->q_raw, n_query++ & 1);
      // 16-byte unit un (8 values) of row qr.
      auto unit = [&](int qr, int un) {
        return *reinterpret_cast<const uint4*>(smem + kOffQ + (un / 8) * kChunk + qr * 128 +
                                               (((un % 8) ^ (qr & 7)) * 16));
      };
#pragma unroll 1
      for (int r0 = 0; r0 < 8; r0 += 2) {
        uint32_t wd[2][8], rd[2][4], top[2] = {0, 0};
        __nv_bfloat162 inv[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int qr = 8 * warp + r0 + r;
          const uint4 v0 = unit(qr, lane), v1 = unit(qr, lane + 32);
          const uint4 vr = kDr && lane < kDr / 8 ? unit(qr, 64 + lane) : make_uint4(0, 0, 0, 0);
          wd[r][0] = v0.x, wd[r][1] = v0.y, wd[r][2] = v0.z, wd[r][3] = v0.w;
          wd[r][4] = v1.x, wd[r][5] = v1.y, wd[r][6] = v1.z, wd[r][7] = v1.w;
          rd[r][0] = vr.x, rd[r][1] = vr.y, rd[r][2] = vr.z, rd[r][3] = vr.w;
          // Largest magnitude of the row: bf16 bits order like their magnitudes.
#pragma unroll
          for (int x = 0; x < 8; ++x) top[r] = max_magnitude2(top[r], wd[r][x]);
          top[r] = larger_half(top[r]);
          if (kDr) {
            uint32_t rope = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) rope = max_magnitude2(rope, rd[r][x]);
            top[r] = max(top[r], rope_magnitude(larger_half(rope)));
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // (The whole warp has read both rows once it has their maxima.)
          top[r] = __reduce_max_sync(0xffffffffu, top[r]);
          const int k = query_exponent(top[r]);
          inv[r] = __float2bfloat162_rn(exp2i(-k));
          if (lane == 0) factor[8 * warp + r0 + r] = exp2i(k);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int qr = 8 * warp + r0 + r;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) split_query(wd[r][4 * e + x], inv[r], &hi[x], &lo[x]);
            const int un = lane + 32 * e;    // 8 codes: half of 16-byte unit (un % 16) / 2
            const int off = (un / 16) * kChunk + qr * 128 + ((((un % 16) >> 1) ^ (qr & 7)) * 16) +
                            (un & 1) * 8;
            *reinterpret_cast<uint2*>(smem + kOffQ + off) =
                make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(smem + kOffQ + 4 * kChunk + off) =
                make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
          }
          if (kDr && lane < kDr / 8) {
            uint32_t o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] = scale_bf16x2(rd[r][x], inv[r]);
            *reinterpret_cast<uint4*>(smem + kOffQ + 8 * kChunk + qr * 128 +
                                      ((lane ^ (qr & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      fence_proxy_async_smem();
      arrive(a_q);
    };

    bool more = seg.next();
    if (more && tid == 0) copy_query(seg.cur);
    if (more) write_query();
    while (more) {
      const int b = seg.cur;
      const int64_t lo = seg.lo, hi = seg.hi, L = seg.L;
      PageWalk walk(pm, page_scales, b, lo, hi);
      int next_b = -1;     // thread 0: the next sequence; its query block into L2 ahead of its use
      if (tid == 0) {
        Segments ahead = seg;
        if (ahead.next()) {
          next_b = ahead.cur;
          const int64_t r0 = int64_t(ahead.cur) * H + g * kHeadsPerCta;
          const int rows = min(H - g * kHeadsPerCta, kHeadsPerCta);
          if (rows > 0) bulk_prefetch_l2(q_cat + r0 * R, uint32_t(rows * R * 2));
        }
      }
      meet_all();                                      // every row's factor is written
      const float row_scale = s_row[((n_query - 1) & 1) * 64 + row] * scale_log2;
      float ref = 0.f, top = -INFINITY, l_sum = 0.f;   // ref: set by the first tile
      for (int64_t t = lo; t < hi; t += 2, ++i) {
        const int sb = i & 1;
        await(&bars->s_full[sb], (i >> 1) & 1);
        // With this sequence's last scores its query block is free.
        if (next_b >= 0 && t + 2 >= hi && ok) copy_query(next_b);
        tc_fence_after();
        uint32_t x[32];          // keys 32 part .. of the page
        tmem_ld32(lanes + kColS + uint32_t(sb) * 64u + uint32_t(part) * 32u, x);
        int64_t unused;
        float sc;                // the page's scale (1 where there is no page)
        walk.at(t + pg, &unused, &sc);
        tmem_wait_ld();
        tc_fence_before();
        arrive(sb ? a_s1 : a_s0);

        const int64_t left = t + pg < hi ? L - (t + pg) * kTileKeys : 0;
        const int valid = int(min(left, int64_t(kTileKeys))) - 32 * part;
        if (valid < 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= valid) x[j] = 0xFF800000u;        // -inf
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(x[j]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        const float f = score_factor(row_scale, sc), lsc = log2f(sc);
        float mt = mx * f + lsc;                        // log2 of the largest p * scale
        float* s_part = s_max + sb * 4 * 64 + row;      // [4 parts][64 rows]
        s_part[(2 * pg + part) * 64] = mt;
        meet();
        mt = fmaxf(fmaxf(s_part[0], s_part[64]), fmaxf(s_part[128], s_part[192]));

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
        const float shift = lsc + kPScale - ref;
        uint32_t hi8[8], lo8[8];
        const float sum = split_probabilities(x, f, shift, hi8, lo8);
        l_sum = fmaf(sum, 1.f / sc, l_sum);

        if (t != lo && __any_sync(0xffffffffu, alpha != 1.f)) {
          await(&bars->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);   // O holds P.C(i - 1)
          tc_fence_after();
#pragma unroll 1
          for (int c = 128 * part; c < 128 * part + 128; c += 64) {
            uint32_t r[2][32];
            tmem_ld32(lanes + kColO + uint32_t(c), r[0]);
            tmem_ld32(lanes + kColO + uint32_t(c) + 32u, r[1]);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; ++e)
              r[e / 32][e % 32] = __float_as_uint(__uint_as_float(r[e / 32][e % 32]) * alpha);
            tmem_st32(lanes + kColO + uint32_t(c), r[0]);
            tmem_st32(lanes + kColO + uint32_t(c) + 32u, r[1]);
          }
          tmem_wait_st();
        }
        // This thread's page of the pair, if there is one: its P tile is free
        // once the product that read it last is done.
        const uint32_t vp = v + uint32_t(pg);
        const int ps = vp % kVStages;
        // Without one, the tile before last must be through: this warp's word for
        // this tile must not count for that one while the other CTA's is on its way.
        if (t + pg < hi) {
          if (vp >= kVStages) await(&bars->vempty[ps], (vp / kVStages - 1) & 1);
        } else if (i >= 2) {
          await(&bars->pv_done[sb], ((i >> 1) - 1) & 1);
        }
        if (t + pg < hi) {
          uint8_t* prow = smem + kOffP + ps * kChunk + row * 128;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int un = part * 2 + u;
            *reinterpret_cast<uint4*>(prow + (un ^ (row & 7)) * 16) =
                make_uint4(hi8[4 * u], hi8[4 * u + 1], hi8[4 * u + 2], hi8[4 * u + 3]);
            *reinterpret_cast<uint4*>(prow + ((un + 4) ^ (row & 7)) * 16) =
                make_uint4(lo8[4 * u], lo8[4 * u + 1], lo8[4 * u + 2], lo8[4 * u + 3]);
          }
        }
        // Rows past the sequence's end may hold anything, NaN codes among it:
        // their weight is 0, so they are zeroed in the staged page.
#pragma unroll 1
        for (int p = 0; p < 2 && t + p < hi; ++p, ++v) {
          const int64_t rows = L - (t + p) * kTileKeys;
          if (rows >= kTileKeys) continue;
          const int vs = v % kVStages;
          await(&bars->vfull[vs], (v / kVStages) & 1);
          uint8_t* stage = smem + kOffV + vs * kVBytes;
          for (int u = tid; u < (kTileKeys - int(rows)) * 16; u += kSoftmaxThreads)
            *reinterpret_cast<uint4*>(stage + (u & 1) * kChunk + (int(rows) + u / 16) * 128 +
                                      ((u / 2) % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        arrive(sb ? a_p1 : a_p0);
      }
      more = seg.next();
      if (more) write_query();
      // Epilogue: normalised partial output and log-sum-exp.
      // The four parts' sums meet in the buffer that the last tile did not use
      // (some warp may still be reading the other; the next sequence's first
      // meeting frees this one).
      float* s_sum = s_max + (i & 1) * 4 * 64 + row;
      s_sum[(2 * pg + part) * 64] = l_sum;
      meet();
      const float l_row = (s_sum[0] + s_sum[64]) + (s_sum[128] + s_sum[192]);
      await(&bars->pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1);
      tc_fence_after();
      const float inv = 1.f / l_row;
      const int slot = b + w;
      // Partials are o_part[slot][d_c / 4][H][4]: a warp stores 32 consecutive
      // heads of one 4-column group (512 contiguous bytes), kept in L2 for the
      // combine that reads them next.
      const uint64_t keep = l2_policy_evict_last();
      // Accumulator column c of product h = c / 128 is latent column
      // 256 h + 128 pg + c % 128.
      float* dst = o_part + ((int64_t(slot) * (kDc / 4) + part * 64 + pg * 32) * H + head) * 4;
      const int64_t step = int64_t(H) * 4;
#pragma unroll 1
      for (int c = 0; c < 128; c += 64) {
        uint32_t r[2][32];
        tmem_ld32(lanes + kColO + uint32_t(128 * part + c), r[0]);
        tmem_ld32(lanes + kColO + uint32_t(128 * part + c + 32), r[1]);
        tmem_wait_ld();
        if (head < H) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint32_t* q = r[e / 8] + 4 * (e % 8);
            st_global_f4_hint(dst, make_float4(__uint_as_float(q[0]) * inv,
                                               __uint_as_float(q[1]) * inv,
                                               __uint_as_float(q[2]) * inv,
                                               __uint_as_float(q[3]) * inv), keep);
            dst += step;
          }
        }
      }
      if (pg == 0 && part == 0 && head < H)
        lse_part[int64_t(slot) * H + head] = (log2f(l_row) + ref - kPScale) * 0.69314718055994531f;
      tc_fence_before();
      arrive(a_o);
    }
    if (tid == 0 && n_copied) {   // the last copy has landed, after a give-up as well
      volatile int no_abort = 0;
      mbar_wait(&bars->q_raw, (n_copied - 1) & 1, &no_abort, kWaitLimitCycles / 100);
    }
  }
  if (!ok && lane == 0) raise_abort(bars, status);

  // Every role has stopped.  The loads that this CTA issued land before its
  // shared memory is released (after a give-up some were never waited for), and
  // neither CTA leaves while the other's products may still read from it.
  __syncwarp();
  if (lane == 0 && (warp == kKWarp || warp == kVWarp)) {
    volatile int no_abort = 0;
    const uint32_t n_st = warp == kKWarp ? kKStages : kVStages;
    for (uint32_t k = (n_issued > n_st ? n_issued - n_st : 0); k < n_issued; ++k)
      mbar_wait(warp == kKWarp ? &bars->kfull[k % n_st] : &bars->vfull[k % n_st], (k / n_st) & 1,
                &no_abort, kWaitLimitCycles / 100);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <int kDr, typename... Args>
cudaError_t launch_t(dim3 grid, cudaStream_t stream, Args... args) {
  static bool attr_done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode8_kernel<kDr>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(kSmemBytes));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl(decode8_kernel<kDr>, grid, dim3(kThreads), kSmemBytes, stream, args...);
}

inline int head_pairs(int H) { return (H + 2 * kHeadsPerCta - 1) / (2 * kHeadsPerCta); }

}  // namespace

// The kernel for up to 64 heads (k_decode_fp8_paged64.cu).
cudaError_t launch_decode_fp8_paged64(const CUtensorMap& tm_codes, const CUtensorMap& tm_rope,
                                      const CUtensorMap& tm_query, const __nv_bfloat16* q_cat, const float* page_scales,
                                      const PageMap& pm, const int32_t* seqlens, int B, int H,
                                      int d_r, int64_t cap, float scale_log2, int W, float* o_part,
                                      float* lse_part, int* status, uint64_t inject_wait,
                                      cudaStream_t stream);

int decode_fp8_paged_splits(int sms, int H) {
  if (H <= kHeadsPerCta) return sms;
  const int W = sms / (2 * head_pairs(H));
  return W < 1 ? 1 : W;
}

cudaError_t launch_decode_fp8_paged(const __nv_bfloat16* q_cat, const uint8_t* pool,
                                    const float* page_scales, const PageMap& pm,
                                    const int32_t* seqlens, int B, int H, int d_r, int64_t cap,
                                    float scale, int W, float* o_part, float* lse_part,
                                    int* status, uint64_t inject_wait, cudaStream_t stream) {
  const uint64_t rows = uint64_t(pm.total_rows(B)), row_bytes = kDc + 2 * d_r;
  CUtensorMap tm_codes, tm_rope;
  if (!make_code_map(&tm_codes, pool, rows, row_bytes)) return cudaErrorInvalidValue;
  tm_rope = tm_codes;
  // The same rows viewed as bf16: the RoPE keys are columns 256 .. 319.
  CUtensorMap tm_query;
  if (!make_map16(&tm_query, q_cat, uint64_t(B) * H, uint64_t(kDc + d_r), uint64_t(kDc + d_r), 64))
    return cudaErrorInvalidValue;
  if (d_r && !make_map16(&tm_rope, pool, rows, row_bytes / 2, row_bytes / 2, kTileKeys))
    return cudaErrorInvalidValue;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (H <= kHeadsPerCta)   // a pair's second CTA would have no heads
    return launch_decode_fp8_paged64(tm_codes, tm_rope, tm_query, q_cat, page_scales, pm, seqlens, B, H, d_r,
                                     cap, scale_log2, W, o_part, lse_part, status, inject_wait,
                                     stream);
  const dim3 grid(2 * head_pairs(H), W);
  auto launch = d_r ? launch_t<64, CUtensorMap, CUtensorMap, CUtensorMap, const float*, PageMap,
                               const __nv_bfloat16*, const int32_t*, int, int, int64_t, float, int,
                               float*, float*, int*, uint64_t>
                    : launch_t<0, CUtensorMap, CUtensorMap, CUtensorMap, const float*, PageMap,
                               const __nv_bfloat16*, const int32_t*, int, int, int64_t, float, int,
                               float*, float*, int*, uint64_t>;
  return launch(grid, stream, tm_codes, tm_rope, tm_query, page_scales, pm, q_cat, seqlens, B, H, cap,
                scale_log2, W, o_part, lse_part, status, inject_wait);
}

}  // namespace mla
