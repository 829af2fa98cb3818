// One serving step's bookkeeping from request lengths: token offsets, pages
// taken from the free list, block-table entries, positions, slots, and the
// runs that the append kernel writes.
//
// Per request b with c cached and t new tokens and pages of P tokens:
//   pages taken     ceil((c + t) / P) - ceil(c / P)
//   pages written   t ? (c + t - 1) / P - c / P + 1 : 0   (its runs)
// Exclusive sums of t, pages taken and runs over the requests place everything
// else: token i of request b sits at position c + i, in a listed page or in the
// j-th page that the request takes.
//
// Bound: latency (16 requests 3.0 us, 256 with 12K new tokens 4.6 us). Every CTA
// scans all requests for itself (a few KB) and fills its share of the outputs, so
// one launch does without a second pass; the last CTA to finish writes kv_len and
// free_next, which may be the buffers that the others read.
#include "kv8_kernels.cuh"
#include "star_common.cuh"
#include "star_kernels.cuh"

namespace star {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Sums {
  long long tok, page, run;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.tok + b.tok, a.page + b.page, a.run + b.run};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, a.tok, d), __shfl_up_sync(0xffffffffu, a.page, d),
              __shfl_up_sync(0xffffffffu, a.run, d)};
}

// Last b with off[b] <= i (off ascending, off[0] = 0 <= i < off[B]).
__device__ __forceinline__ int owner(const int* off, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(kThreads) batch_plan_kernel(const __grid_constant__ BatchPlanParams p) {
  extern __shared__ int sm[];
  int* tok = sm;                 // [B + 1] exclusive sums
  int* page = tok + p.B + 1;
  int* run = page + p.B + 1;
  int* ctx = run + p.B + 1;      // [B]
  __shared__ Sums warp_sum[kWarps];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  after_previous();
  const int P = 1 << p.page_shift;
  const long long limit = static_cast<long long>(p.max_pages) << p.page_shift;

  // each thread sums a contiguous part of the requests
  const int per = ceil_div(p.B, kThreads);
  const int b0 = imin(p.B, tid * per), b1 = imin(p.B, b0 + per);
  Sums mine{0, 0, 0};
  int bad = 0;
  auto request = [&](int b, long long& c, long long& t) -> Sums {
    c = p.ctx_len[b];
    t = p.new_len[b];
    if (c < 0 || t < 0 || c + t > limit) {
      bad = 1;
      t = 0;
      if (c < 0) c = 0;
    }
    return Sums{t, ((c + t + P - 1) >> p.page_shift) - ((c + P - 1) >> p.page_shift),
                t ? ((c + t - 1) >> p.page_shift) - (c >> p.page_shift) + 1 : 0};
  };
  for (int b = b0; b < b1; ++b) {
    long long c, t;
    mine = mine + request(b, c, t);
  }
  const int begin = *p.free_begin;
  Sums inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums up = shfl_up(inc, d);
    if (lane >= d) inc = inc + up;
  }
  if (lane == 31) warp_sum[warp] = inc;
  bad = __syncthreads_or(bad);
  Sums base{0, 0, 0}, total{0, 0, 0};
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) base = total;
    total = total + warp_sum[w];
  }
  if (begin < 0 || total.tok > p.n_cap || total.page > static_cast<long long>(p.num_free) - begin) bad = 1;
  // a step that does not fit is refused as a whole: every thread of every CTA
  // comes to the same answer
  const int n = bad ? 0 : static_cast<int>(total.tok);
  const int pages = bad ? 0 : static_cast<int>(total.page);
  const int runs = bad ? 0 : static_cast<int>(total.run);
  Sums at = base + Sums{inc.tok - mine.tok, inc.page - mine.page, inc.run - mine.run};
  for (int b = b0; b < b1; ++b) {
    long long c, t;
    const Sums s = request(b, c, t);
    tok[b] = bad ? 0 : static_cast<int>(at.tok);
    page[b] = bad ? 0 : static_cast<int>(at.page);
    run[b] = bad ? 0 : static_cast<int>(at.run);
    ctx[b] = static_cast<int>(c);
    at = at + s;
  }
  if (tid == 0) {
    tok[p.B] = n;
    page[p.B] = pages;
    run[p.B] = runs;
  }
  __syncthreads();

  const int stride = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
  for (int i = first; i < p.n_cap; i += stride) {
    int at_pos = 0, slot = -1;
    if (i < n) {
      const int b = owner(tok, p.B, i), c = ctx[b];
      at_pos = c + i - tok[b];
      const int j = at_pos >> p.page_shift, listed = (c + P - 1) >> p.page_shift;
      const int id = j < listed ? p.table[static_cast<size_t>(b) * p.max_pages + j]
                                : p.free_pages[begin + page[b] + j - listed];
      const int row = at_pos & (P - 1);
      // a listed page outside int32 slots is the caller's mistake, not a row
      const bool fits = id >= 0 && id <= (INT32_MAX >> p.page_shift);
      if (!fits) atomicOr(p.status, kDevBounds);
      slot = fits ? (id << p.page_shift) + row : -1;
      if (i == tok[b] || row == 0) p.run_start[run[b] + j - (c >> p.page_shift)] = i;
    }
    p.pos[i] = at_pos;
    p.slot[i] = slot;
  }
  for (int i = first; i < pages; i += stride) {
    const int b = owner(page, p.B, i);
    const int j = ((ctx[b] + P - 1) >> p.page_shift) + i - page[b];
    p.table[static_cast<size_t>(b) * p.max_pages + j] = p.free_pages[begin + i];
  }
  for (int i = runs + first; i <= p.run_cap; i += stride) p.run_start[i] = n;
  for (int b = first; b <= p.B; b += stride) p.cu_new[b] = tok[b];

  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) last = inc_acq_rel(p.ticket, gridDim.x - 1) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
  }
  for (int b = tid; b < p.B; b += kThreads) {
    const int t = tok[b + 1] - tok[b];
    // a refused step leaves the lengths as they were, valid or not
    p.kv_len[b] = bad ? p.ctx_len[b] : ctx[b] + t;
  }
  if (tid == 0) {
    *p.free_next = begin + pages;
    if (bad) atomicOr(p.status, kDevBounds);
  }
}

cudaError_t launch_batch_plan(const BatchPlanParams& p, cudaStream_t stream) {
  const size_t smem = (4 * static_cast<size_t>(p.B) + 3) * sizeof(int);
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = set_smem_attr_once((const void*)batch_plan_kernel, 10, dev,
                                     (4 * kMaxRequests + 3) * sizeof(int));
  if (e != cudaSuccess) return e;
  // An output a thread (256 requests, 12K tokens: 4.6 us; four outputs, or 512
  // threads: 6.7 and 5.1 us). One CTA needs no ticket.
  const int most = imax(p.n_cap, p.run_cap);
  const int grid = imax(1, imin(148, ceil_div(most, kThreads)));
  return launch_after(batch_plan_kernel, dim3(grid), kThreads, smem, stream, p);
}

}  // namespace star
