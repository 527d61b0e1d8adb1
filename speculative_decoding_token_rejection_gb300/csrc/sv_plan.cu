// sv_plan.cu -- block tables, positions and slots of a step from request lengths.
//
// Everything is whole numbers and a few bytes a row, so what counts is the chain
// of dependent steps: three prefix sums over the requests (rows, pages wanted,
// pages given back), then every row finds its request.  One CTA does the sums
// and the requests' outputs, 1024 requests at a time; a row's request is the
// last one that begins at or before it, found by writing requests to the places
// where they begin and taking a running maximum.  A small step's rows, and the
// pages given back, are the same CTA's work, otherwise a second kernel's:
// kRowsCta rows or kBackCta requests a CTA.
//
// Bound by latency.  4 requests x 5 rows: 5.9 us for the launch and the chain
// (7.2 as two kernels); 512 requests that hold 512 pages each, 2700 rows, a
// tenth done: 9.7 us (26 in one CTA); 64 prompts, 0.5 million rows: 12.0 us;
// 4096 requests: 18.0 us.  One CTA is the faster up to 250 requests of 64
// pages (6.8 us against 9.0) or 16 of 1024 (7.8, 8.0; 32: 10.3 against 8.0).
//
// A page newly given to a request is written to its table by the row of the
// page's first token, which has just read it from the ring.  (There is one: the
// pages held before hold all computed tokens, so a new page begins with a new one.)
#include <cstdint>

#include "sv_internal.h"
#include "sv_ops.cuh"

namespace sv {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kRowsCta = 1024;      // rows of a CTA of the second kernel, and of a step of the first
constexpr int kRowsThreads = 256;
constexpr int kBackCta = 4;         // requests of a CTA of the second kernel that gives pages back
constexpr int kRowsOne = 2048;      // rows that one CTA does by itself
constexpr int64_t kPagesOne = 20480;  // and block table entries, which may all be given back

struct Workspace {  // of every request
  int32_t *end;    // its last row + 1 (at most R)
  int32_t *start;  // place in the ring of the first page it is given; ~place of the first it gives back
  int32_t *held;   // pages held before
};
__device__ __forceinline__ Workspace workspace_of(const PlanParams &P) {
  int32_t *w = static_cast<int32_t *>(P.workspace);
  return Workspace{w, w + P.N, w + 2 * static_cast<int64_t>(P.N)};
}

struct Sums {
  int64_t rows, want, back;
};
__device__ __forceinline__ Sums warp_scan(Sums x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b < 32; b <<= 1) {
    const Sums y{__shfl_up_sync(0xFFFFFFFFu, x.rows, b), __shfl_up_sync(0xFFFFFFFFu, x.want, b),
                 __shfl_up_sync(0xFFFFFFFFu, x.back, b)};
    if (lane >= b) x = Sums{x.rows + y.rows, x.want + y.want, x.back + y.back};
  }
  return x;
}

// Rows [r0, r0 + kRowsCta) by THREADS threads; requests i0 .. i1 are all that have rows there, and r0's is among them.
template <int THREADS>
__device__ __forceinline__ void do_rows(const PlanParams &P, const Workspace &W, int r0, int i0, int i1, int32_t *mark,
                                        int32_t *warp_last) {
  constexpr int kPer = kRowsCta / THREADS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();  // (the step before is done with the marks)
#pragma unroll
  for (int k = 0; k < kPer; ++k) mark[k * THREADS + tid] = -1;
  __syncthreads();
  for (int i = i0 + tid; i <= i1; i += THREADS) {
    const int first = i ? W.end[i - 1] : 0;
    // (of those that begin at one row the last is the one that has rows)
    if (first < r0 + kRowsCta && W.end[i] > r0) atomicMax(&mark[max(0, first - r0)], i);
  }
  __syncthreads();
  // the running maximum, kPer neighbouring rows a thread
  int req[kPer], most = -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) req[k] = most = max(most, mark[tid * kPer + k]);
  int up = most;
#pragma unroll
  for (int b = 1; b < 32; b <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, up, b);
    if (lane >= b) up = max(up, y);
  }
  if (lane == 31) warp_last[warp] = up;
  __syncthreads();
  int before = __shfl_up_sync(0xFFFFFFFFu, up, 1);
  if (lane == 0) before = -1;
  for (int w = 0; w < warp; ++w) before = max(before, warp_last[w]);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t row = static_cast<int64_t>(r0) + tid * kPer + k;
    if (row >= P.R) break;
    const int i = max(req[k], before);
    int pos = -1;
    int64_t slot = -1;
    if (i >= 0 && row < W.end[i] && P.seq_lens[i] > 0) {
      const int seq = P.seq_lens[i], held = W.held[i];
      pos = seq - static_cast<int>(W.end[i] - row);
      const int x = div_by(pos, P.page);
      int32_t *const entry = P.tables + i * P.table_stride + x;
      int page;
      if (x < held) {
        page = *entry;
      } else {
        const int64_t at = static_cast<int64_t>(W.start[i]) + x - held;
        page = P.ring[at < P.capacity ? at : at - P.capacity];
        if (pos == x * P.block) *entry = page;
      }
      slot = static_cast<int64_t>(page) * P.block + (pos - x * P.block);
    }
    P.positions[row] = pos;
    P.slots[row] = slot;
  }
}

// The first request whose rows end behind `row` (N: none), by all lanes of a warp: 32 places at a time.
__device__ __forceinline__ int request_behind(const int32_t *end, int n, int64_t row) {
  int lo = 0, hi = n;  // it is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, at = lo + static_cast<int>(threadIdx.x & 31) * step;
    const uint32_t behind = __ballot_sync(0xFFFFFFFFu, at >= hi || end[at] > row);
    const int k = behind ? __ffs(behind) - 1 : 32;  // (requests are in order: all lanes from k on)
    if (k < 32) hi = min(hi, lo + k * step);
    if (k > 0) lo += (k - 1) * step + 1;
  }
  return lo;
}

// The pages of a request that is done go to the places behind the ring's end, by `threads` threads.
__device__ __forceinline__ void give_back(const PlanParams &P, const Workspace &W, int i, int thread, int threads) {
  if (W.start[i] >= 0) return;
  const int64_t to = ~W.start[i];
  const int count = W.held[i] - P.shared;
  const int32_t *const row = P.tables + i * P.table_stride + P.shared;
#pragma unroll 8
  for (int k = thread; k < count; k += threads) {
    const int64_t at = to + k;  // (below twice the capacity: there is room for them)
    P.ring[at < P.capacity ? at : at - P.capacity] = row[k];
  }
}

template <bool ROWS>
__global__ void __launch_bounds__(kPlanThreads) plan_requests_kernel(const PlanParams P) {
  pdl_enter();
  __shared__ Sums warp_sums[kPlanWarps];
  __shared__ int32_t mark[ROWS ? kRowsCta : 1], warp_last[kPlanWarps];
  __shared__ unsigned long long given, returned;  // pages
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Workspace W = workspace_of(P);
  const int64_t head = P.range[0], tail = P.range[1];
  uint32_t bits = 0;
  const bool pool = head >= 0 && tail >= head && tail - head <= P.capacity;
  if (!pool) bits |= SV_DATA_BAD_PARAM;
  const int64_t from = pool ? head % P.capacity : 0, to = pool ? tail % P.capacity : 0;
  // (places behind the tail: what goes there meets no page that is being taken)
  const int64_t room = pool ? P.capacity - (tail - head) : 0;
  if (tid == 0) given = returned = 0;
  Sums before{0, 0, 0};  // of the steps before
  for (int base = 0; base < P.N; base += kPlanThreads) {
    const int i = base + tid;
    const bool in = i < P.N;
    int64_t n = in ? P.fresh[i] : 0;
    const int64_t p = in ? P.computed[i] : 0;
    const int held = in ? P.held[i] : 0;
    const bool done = p < 0, holds = held >= 0 && held <= P.width;
    bool good = in && !done;
    if (n < 0 || !holds) {
      good = false;
      bits |= SV_DATA_BAD_PARAM;
    }
    if (n < 0) n = 0;
    const int64_t len = p + n;
    const uint32_t pages = static_cast<uint32_t>(len) / static_cast<uint32_t>(P.block);  // (both counts are below 2^31)
    const int64_t need = pages + (pages * static_cast<uint32_t>(P.block) != static_cast<uint32_t>(len));
    if (good && (need > P.width || len > 0x7FFFFFFF || static_cast<int64_t>(held) * P.block < p || held < P.shared)) {
      good = false;
      bits |= SV_DATA_BAD_PARAM;
    }
    const int64_t want = good && need > held ? need - held : 0;
    const bool gone = in && done && pool && holds && held > P.shared;
    const int back = gone ? held - P.shared : 0;
    Sums x = warp_scan(Sums{n, want, back});
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = warp_scan(warp_sums[lane]);
    __syncthreads();
    if (warp > 0) {
      const Sums y = warp_sums[warp - 1];
      x = Sums{x.rows + y.rows, x.want + y.want, x.back + y.back};
    }
    x = Sums{x.rows + before.rows, x.want + before.want, x.back + before.back};
    const Sums step = warp_sums[kPlanWarps - 1];
    before = Sums{before.rows + step.rows, before.want + step.want, before.back + step.back};
    // (requests whose rows do not fit are the last ones: what they want is nobody's loss)
    if (good && x.rows > P.R) {
      good = false;
      bits |= SV_DATA_BAD_CU;
    }
    if (good && want > 0 && (!pool || x.want > tail - head)) {
      good = false;
      bits |= SV_DATA_NO_PAGES;
    }
    const bool returns = gone && x.back <= room;
    if (gone && !returns) bits |= SV_DATA_BAD_PARAM;
    const bool takes = good && want > 0;
    if (in) {
      int64_t place = 0;
      if (takes) place = from + x.want - want;  // (below twice the capacity)
      W.end[i] = static_cast<int32_t>(min(x.rows, P.R));
      W.start[i] = returns ? ~static_cast<int32_t>((to + x.back - back) % P.capacity)
                           : static_cast<int32_t>(place < P.capacity ? place : place - P.capacity);
      W.held[i] = held;
      if (P.cu) P.cu[i] = static_cast<int32_t>(min(x.rows - (i + 1), int64_t{0x7FFFFFFF}));
      P.held_out[i] = returns ? P.shared : takes ? static_cast<int32_t>(need) : held;
      P.seq_lens[i] = good ? static_cast<int32_t>(len) : 0;
    }
    if (takes) atomicMax(&given, static_cast<unsigned long long>(x.want));
    if (returns) atomicMax(&returned, static_cast<unsigned long long>(x.back));
    __syncthreads();  // (the sums have been read, and the outputs are there)
  }
  if (P.N == 0) __syncthreads();
  if (tid == 0) {
    P.range_out[0] = head + static_cast<int64_t>(given);
    P.range_out[1] = tail + static_cast<int64_t>(returned);
  }
  if (P.status) {
    bits = __reduce_or_sync(0xFFFFFFFFu, bits);
    if (lane == 0 && bits) atomicOr(P.status, static_cast<int>(bits));
  }
  if (ROWS) {
    int warps = 1;  // of a request
    while (warps < kPlanWarps && warps * P.N < kPlanWarps) warps *= 2;
    const int at_once = kPlanWarps / warps;
    for (int i = warp % at_once; i < P.N; i += at_once) give_back(P, W, i, (warp / at_once) * 32 + lane, warps * 32);
    for (int r0 = 0; r0 < P.R; r0 += kRowsCta) do_rows<kPlanThreads>(P, W, r0, 0, P.N - 1, mark, warp_last);
  }
}

// The first `rows_ctas` CTAs take rows, the others requests that give pages back.
__global__ void __launch_bounds__(kRowsThreads) plan_rows_kernel(const PlanParams P, int rows_ctas) {
  pdl_enter();
  __shared__ int32_t mark[kRowsCta], warp_last[kRowsThreads / 32], range[2];
  const Workspace W = workspace_of(P);
  if (static_cast<int>(blockIdx.x) >= rows_ctas) {
    const int first = (blockIdx.x - rows_ctas) * kBackCta;
    for (int i = first; i < min(first + kBackCta, P.N); ++i) give_back(P, W, i, threadIdx.x, kRowsThreads);
    return;
  }
  const int r0 = blockIdx.x * kRowsCta, warp = threadIdx.x >> 5;
  if (warp < 2) {
    const int i = request_behind(W.end, P.N, warp ? min(r0 + static_cast<int64_t>(kRowsCta), P.R) - 1 : r0);
    if ((threadIdx.x & 31) == 0) range[warp] = warp ? min(i, P.N - 1) : i;
  }
  __syncthreads();
  do_rows<kRowsThreads>(P, W, r0, range[0], range[1], mark, warp_last);
}

}  // namespace

int64_t plan_workspace_bytes(int32_t n) { return 12 * static_cast<int64_t>(n) + 16; }

cudaError_t launch_plan(const PlanParams &p, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg{};
  const bool one = p.R <= kRowsOne && static_cast<int64_t>(p.N) * (p.width + 1) <= kPagesOne;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = launch_attrs(attr, 0, p.pdl);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, one ? plan_requests_kernel<true> : plan_requests_kernel<false>, p);
  if (e != cudaSuccess || one) return e;
  const int64_t rows = (static_cast<int64_t>(p.R) + kRowsCta - 1) / kRowsCta;
  cfg.gridDim = dim3(static_cast<unsigned>(rows + (static_cast<int64_t>(p.N) + kBackCta - 1) / kBackCta));
  cfg.blockDim = dim3(kRowsThreads);
  return cudaLaunchKernelEx(&cfg, plan_rows_kernel, p, static_cast<int>(rows));
}

}  // namespace sv
