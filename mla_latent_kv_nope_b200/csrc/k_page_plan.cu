// Page plans: block tables, slot maps and positions of one serving step, built
// on the device from the requests' lengths, and the return of finished
// requests' pages.
//
// Request b holds L_b tokens and adds n_b.  With pages(L) = ceil(L / 64) it
// needs pages(L_b + n_b) - pages(L_b) new pages, popped off the end of the free
// list in request order; token i of request b sits at position L_b + i.
//
// Whole numbers only: bound by latency for a decode step and by the 12 bytes
// written per token for prompts.  One launch: every block walks the request
// lengths (a few KB out of L2) and forms the two prefix sums itself, 256
// requests at a time, then expands its own slice of the tokens and of the new
// pages, so no block waits for another.  Only where the lengths or the free count are
// updated in place are they left to the block that finishes last.  Measured on B200:
// 64 sequences, one token each, 3.5 us; 256 prompts of 65,900 tokens 4.3 us, in place
// 5.6 (7.1 with 1024 tokens a block and one reduction per total).
#include "kernels.h"

namespace mla {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanTokens = 512;    // tokens per block

__device__ __forceinline__ int64_t pages_of(int64_t L) { return (L + kTileKeys - 1) / kTileKeys; }

// Sums over the block of two 64-bit values, and whether any thread's `bad` is
// set (every thread gets them; one barrier).
__device__ __forceinline__ void block_sum2(int64_t& a, int64_t& b, int& bad,
                                           int64_t (*red)[2]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][0] = a, red[threadIdx.x >> 5][1] = b;
  bad = __syncthreads_or(bad);
  a = b = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) a += red[w][0], b += red[w][1];
}

// Inclusive prefix over the block of two values (one barrier).
__device__ __forceinline__ void block_scan2(int32_t& a, int32_t& b, int32_t (*red)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t ua = __shfl_up_sync(0xffffffffu, a, o), ub = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) a += ua, b += ub;
  }
  if (lane == 31) red[warp][0] = a, red[warp][1] = b;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w)
    if (w < warp) a += red[w][0], b += red[w][1];
}

// Smallest i in [0, n) with end[i] > v (end ascending; the caller knows one exists).
__device__ __forceinline__ int first_past(const int32_t* end, int n, int32_t v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > v) hi = mid; else lo = mid + 1;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* seqlens;
  const int32_t* new_lens;
  int B;
  int32_t* block_table;
  int max_blocks;
  int64_t capacity;         // the longest sequence, at most 64 * max_blocks < 2^31
  const int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int64_t num_pages;
  int T;
  int32_t* query_start;
  int32_t* positions;
  int64_t* slots;
  int32_t* token_request;   // or null
  int32_t* seqlens_out;
  int32_t* free_count_out;
  uint32_t* ticket;
  bool in_place;            // seqlens_out is seqlens or free_count_out is free_count
  int page_slice;           // new pages per block
  int* status;
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs a) {
  __shared__ int64_t s_red[kPlanThreads / 32][2];
  __shared__ int32_t s_red2[kPlanThreads / 32][2];
  __shared__ int32_t s_tok[kPlanThreads], s_page[kPlanThreads];   // ends of each request's share
  __shared__ int32_t s_len[kPlanThreads], s_new[kPlanThreads];
  __shared__ bool s_last;
  const int tid = threadIdx.x;
  pdl_wait();
  const int32_t free_n = *a.free_count;

  // Totals and checks: a step that cannot be served as a whole is not begun.
  // The first kPlanThreads requests stay in registers for the second walk.
  int64_t tok = 0, need = 0;
  int bad = 0;
  int32_t L0 = 0, n0 = 0;
  for (int b = tid; b < a.B; b += kPlanThreads) {
    const int32_t Lb = a.seqlens[b], nb = a.new_lens[b];
    if (b == tid) L0 = Lb, n0 = nb;
    const int64_t L = Lb, n = nb;
    if (L < 0 || n < 0 || L + n > a.capacity) bad = 1;
    else tok += n, need += pages_of(L + n) - pages_of(L);
  }
  block_sum2(tok, need, bad, s_red);
  if (tok > a.T || need > free_n || free_n < 0 || free_n > a.free_capacity) bad = 1;
  if (bad) tok = need = 0;

  const int32_t t0 = int32_t(blockIdx.x) * kPlanTokens, t1 = min(t0 + kPlanTokens, a.T);
  const int32_t live1 = int32_t(min(int64_t(t1), tok));           // end of this block's live tokens
  const int64_t p0 = int64_t(blockIdx.x) * a.page_slice;
  const int64_t p1 = min(p0 + a.page_slice, need);
  int page_bad = 0;
  int32_t tok_base = 0, page_base = 0;
  for (int b0 = 0; b0 < a.B && !bad; b0 += kPlanThreads) {
    // Block 0 writes query_start for every request, so it walks them all.
    if (blockIdx.x && tok_base >= live1 && page_base >= p1) break;
    const int b = b0 + tid;
    const bool in_regs = b0 == 0;
    const int32_t L = in_regs ? L0 : b < a.B ? a.seqlens[b] : 0;
    const int32_t n = in_regs ? n0 : b < a.B ? a.new_lens[b] : 0;
    int32_t te = n, pe = int32_t(pages_of(int64_t(L) + n) - pages_of(L));
    block_scan2(te, pe, s_red2);
    te += tok_base, pe += page_base;
    s_tok[tid] = te, s_page[tid] = pe, s_len[tid] = L, s_new[tid] = n;
    if (blockIdx.x == 0 && b < a.B) a.query_start[b + 1] = te;
    __syncthreads();
    const int32_t tok_end = s_tok[kPlanThreads - 1], page_end = s_page[kPlanThreads - 1];
#pragma unroll 4
    for (int32_t t = max(t0, tok_base) + tid; t < min(live1, tok_end); t += kPlanThreads) {
      const int r = first_past(s_tok, kPlanThreads, t);
      const int64_t Lr = s_len[r], have = pages_of(Lr);
      const int64_t pos = Lr + (t - (s_tok[r] - s_new[r])), j = pos / kTileKeys;
      const int32_t first = s_page[r] - int32_t(pages_of(Lr + s_new[r]) - have);
      const int32_t pg = j < have ? a.block_table[int64_t(b0 + r) * a.max_blocks + j]
                                  : a.free_pages[free_n - 1 - (first + int32_t(j - have))];
      const bool ok = pg >= 0 && pg < a.num_pages;
      page_bad |= !ok;
      a.positions[t] = int32_t(pos);
      a.slots[t] = ok ? int64_t(pg) * kTileKeys + pos % kTileKeys : -1;
      if (a.token_request) a.token_request[t] = b0 + r;
    }
    for (int64_t p = max(p0, int64_t(page_base)) + tid; p < min(p1, int64_t(page_end));
         p += kPlanThreads) {
      const int r = first_past(s_page, kPlanThreads, int32_t(p));
      const int64_t end = pages_of(int64_t(s_len[r]) + s_new[r]);   // last new block + 1
      a.block_table[int64_t(b0 + r) * a.max_blocks + end - (s_page[r] - p)] =
          a.free_pages[free_n - 1 - p];
    }
    tok_base = tok_end, page_base = page_end;
    __syncthreads();
  }
  // Rows behind the last request's tokens.
  for (int32_t t = max(t0, int32_t(tok)) + tid; t < t1; t += kPlanThreads) {
    a.positions[t] = -1;
    a.slots[t] = -1;
    if (a.token_request) a.token_request[t] = -1;
  }
  if (blockIdx.x == 0) {
    if (tid == 0) a.query_start[0] = 0;
    if (bad)
      for (int b = tid; b < a.B; b += kPlanThreads) a.query_start[b + 1] = 0;
  }
  if (page_bad || (bad && blockIdx.x == 0 && tid == 0)) record_status(a.status, MLA_ERR_BOUNDS);

  // The lengths and the free count may be updated in place; then they are
  // written once every block has read them, else by the last block in order
  // (256 prompts: 4.3 us without the ticket, 5.6 with it).
  __syncthreads();
  if (tid == 0) {
    bool last = blockIdx.x == gridDim.x - 1;
    if (a.in_place && gridDim.x > 1) {
      __threadfence();
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
      if (last) *a.ticket = 0;
      __threadfence();
    }
    s_last = last;
  }
  __syncthreads();
  if (!s_last) return;
  if (tid < a.B) a.seqlens_out[tid] = L0 + (bad ? 0 : n0);
  for (int b = tid + kPlanThreads; b < a.B; b += kPlanThreads)
    a.seqlens_out[b] = a.seqlens[b] + (bad ? 0 : a.new_lens[b]);
  if (tid == 0) *a.free_count_out = free_n - int32_t(need);
}

constexpr int kReleaseThreads = 1024;

// One block: pages go back to the free list in request and block order.
__global__ void __launch_bounds__(kReleaseThreads)
page_release_kernel(int32_t* seqlens, const int32_t* __restrict__ release, int B,
                    int32_t* block_table, int max_blocks, int32_t* free_pages, int free_capacity,
                    int32_t* free_count, int64_t num_pages, int* status) {
  __shared__ int32_t s_end[kReleaseThreads];
  __shared__ int64_t s_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t cap = int64_t(max_blocks) * kTileKeys;
  pdl_wait();
  if (tid == 0) s_total = 0;
  __syncthreads();
  // Totals and checks first: nothing is returned from a call with a bad page.
  int64_t total = 0;
  int bad = 0;
  for (int b = warp; b < B; b += kReleaseThreads / 32) {
    if (!release[b]) continue;
    const int32_t L = seqlens[b];
    if (L < 0 || L > cap) {
      bad = 1;
      continue;
    }
    const int n = int(tiles_of(L));
    for (int j = lane; j < n; j += 32) {
      const int32_t pg = block_table[int64_t(b) * max_blocks + j];
      if (pg < 0 || pg >= num_pages) bad = 1;
    }
    if (lane == 0) total += n;
  }
  if (total) atomicAdd(reinterpret_cast<unsigned long long*>(&s_total), (unsigned long long)total);
  bad = __syncthreads_or(bad);
  const int32_t held = *free_count;
  if (bad || held < 0 || held + s_total > free_capacity) {
    if (tid == 0) record_status(status, MLA_ERR_BOUNDS);
    return;
  }
  int32_t base = held;
  for (int b0 = 0; b0 < B; b0 += kReleaseThreads) {
    const int b = b0 + tid;
    const int32_t n = (b < B && release[b]) ? int32_t(tiles_of(seqlens[b])) : 0;
    int32_t e = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, e, o);
      if (lane >= o) e += u;
    }
    __shared__ int32_t s_warp[32];
    if (lane == 31) s_warp[warp] = e;
    __syncthreads();
    for (int w = 0; w < warp; ++w) e += s_warp[w];
    s_end[tid] = e;
    __syncthreads();
    for (int r = warp; r < kReleaseThreads && b0 + r < B; r += kReleaseThreads / 32) {
      const int32_t first = r ? s_end[r - 1] : 0, cnt = s_end[r] - first;
      int32_t* row = block_table + int64_t(b0 + r) * max_blocks;
      for (int32_t j = lane; j < cnt; j += 32) {
        free_pages[base + first + j] = row[j];
        row[j] = -1;
      }
    }
    base += s_end[kReleaseThreads - 1];
    if (b < B && release[b]) seqlens[b] = 0;
    __syncthreads();
  }
  if (tid == 0) *free_count = base;
}

}  // namespace

cudaError_t launch_page_plan(const int32_t* seqlens, const int32_t* new_lens, int B,
                             int32_t* block_table, int max_blocks, int64_t capacity,
                             const int32_t* free_pages, int free_capacity,
                             const int32_t* free_count, int64_t num_pages, int T,
                             int32_t* query_start, int32_t* positions, int64_t* slots,
                             int32_t* token_request, int32_t* seqlens_out,
                             int32_t* free_count_out, void* workspace, int* status,
                             cudaStream_t stream) {
  const int grid = T > 0 ? (T + kPlanTokens - 1) / kPlanTokens : 1;
  // A request with n new tokens takes at most n / 64 + 1 new pages.
  const int64_t most = int64_t(T) / kTileKeys + B;
  const PlanArgs a{seqlens, new_lens, B, block_table, max_blocks, capacity, free_pages,
                   free_capacity, free_count, num_pages, T, query_start, positions, slots, token_request,
                   seqlens_out, free_count_out, static_cast<uint32_t*>(workspace),
                   seqlens_out == seqlens || free_count_out == free_count,
                   int((most + grid - 1) / grid), status};
  return launch_pdl(page_plan_kernel, dim3(grid), dim3(kPlanThreads), 0, stream, a);
}

cudaError_t launch_page_release(int32_t* seqlens, const int32_t* release, int B,
                                int32_t* block_table, int max_blocks, int32_t* free_pages,
                                int free_capacity, int32_t* free_count, int64_t num_pages,
                                int* status, cudaStream_t stream) {
  return launch_pdl(page_release_kernel, dim3(1), dim3(kReleaseThreads), 0, stream, seqlens,
                    release, B, block_table, max_blocks, free_pages, free_capacity, free_count,
                    num_pages, status);
}

}  // namespace mla
