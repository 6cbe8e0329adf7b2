// Adapters of many requests beside a shared NF4 projection: the grouping of
// the tokens by adapter, and the projection's kernels.
//
//   y[t] = W x[t] + B[a] p[t],  p[t] = s[a] A[a] x[t]
#include "e4b_device.cuh"
#include "e4b_internal.h"
#include "launch.cuh"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ----------------------------------------------------------------------------
// Grouping: a stable counting sort of the tokens by adapter in one block.
// Every warp owns a contiguous run of tokens and a histogram row of its own in
// shared memory; to place the tokens, lanes with equal ids find one another with a
// warp match, so that the order is fixed.  Two passes over the ids (count, place)
// around one scan over the adapters, thread a owning adapter a.  Latency bounds it
// (one read of the ids and a dozen block-wide steps; 777 tokens of 16 adapters 5 us,
// 8192 of 64 10 us), so the scan's sums go through one barrier and the histogram is
// read once, all warps' rows at a time.
// ----------------------------------------------------------------------------
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;

__global__ void __launch_bounds__(kGroupThreads, 1)
    adapter_group_kernel(const int32_t* __restrict__ ids, int T, int n, int rows_cap, int32_t* __restrict__ order,
                         int32_t* __restrict__ offsets, int32_t* __restrict__ steps) {
  grid_wait();
  grid_launch_dependents();
  extern __shared__ int32_t table[];  // [kGroupWarps][n + 1]
  __shared__ int32_t wsum[2][kGroupWarps];
  __shared__ int32_t none_total;
  __shared__ int32_t first_row[E4B_MAX_ADAPTERS + 1], first_task[E4B_MAX_ADAPTERS + 1];
  __shared__ int32_t last_row[E4B_MAX_ADAPTERS];  // one past an adapter's tokens
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cols = n + 1;
  const int per = ((T + kGroupWarps - 1) / kGroupWarps + 31) / 32 * 32;
  const int t0 = min(T, warp * per), t1 = min(T, t0 + per);
  int32_t* mine = table + warp * cols;
  auto adapter_of = [&](int t) -> int {
    if (t >= t1) return -1;
    const uint32_t a = (uint32_t)__ldg(ids + t);
    return a < (uint32_t)n ? (int)a : n;
  };
  // 256 tokens of a warp at a time: eight loads in flight (one at a time, a warp's 256 tokens took 5 us a pass)
  constexpr int kAhead = 8;
  int ad[kAhead];
  auto load = [&](int tb) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ad[i] = adapter_of(tb + 32 * i + lane);
  };
  load(t0);
  for (int i = lane; i < cols; i += 32) mine[i] = 0;
  __syncwarp();
  for (int tb = t0; tb < t1; tb += 32 * kAhead) {
    if (tb > t0) load(tb);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (ad[i] >= 0) atomicAdd(&mine[ad[i]], 1);  // this warp's row: integers, any order
    }
  }
  __syncthreads();
  // Adapter tid: its tokens in each warp, its padded rows and its 128-row projection tasks.
  int at[kGroupWarps];
  int count = 0;
#pragma unroll
  for (int w = 0; w < kGroupWarps; ++w) {
    const int c = tid < n ? table[w * cols + tid] : 0;
    at[w] = count;
    count += c;
  }
  if (warp == kGroupWarps - 1) {  // the tokens without an adapter: their places, from the end of the adapters' rows
    const int c = table[lane * cols + n];
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    table[lane * cols + n] = x - c;
    if (lane == 31) none_total = x;
  }
  const int padded = (count + kAdapterRowAlign - 1) / kAdapterRowAlign * kAdapterRowAlign;
  const int ntask = (padded + kAdapterTaskRows - 1) / kAdapterTaskRows;
  auto warp_scan = [&](int v) -> int {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  const int in_rows = warp_scan(padded), in_tasks = warp_scan(ntask);
  if (lane == 31) {
    wsum[0][warp] = in_rows;
    wsum[1][warp] = in_tasks;
  }
  __syncthreads();
  auto before = [&](int which, int& total) -> int {  // sum of the warps ahead of this one, and of all
    const int v = wsum[which][lane], x = warp_scan(v);
    total = __shfl_sync(kFull, x, 31);
    return __shfl_sync(kFull, x - v, warp);
  };
  int none0, adapter_tasks;
  const int start = before(0, none0) + in_rows - padded;
  const int task0 = before(1, adapter_tasks) + in_tasks - ntask;
  const int nnone = none_total, none_tasks = (nnone + kAdapterTaskRows - 1) / kAdapterTaskRows;
  const int used = none0 + nnone;
  int32_t* granules = steps + kAdapterStepsHeader;
  int4* tasks = reinterpret_cast<int4*>(steps + adapter_tasks_offset(rows_cap));
  if (tid < n) {  // where each warp's tokens of this adapter start
#pragma unroll
    for (int w = 0; w < kGroupWarps; ++w) table[w * cols + tid] = start + at[w];
  }
  if (tid < n) {
    first_row[tid] = start;
    first_task[tid] = task0;
    last_row[tid] = start + count;
    offsets[tid] = start;
  }
  if (tid == 0) {
    first_row[n] = none0;
    first_task[n] = adapter_tasks;
  }
  __syncthreads();
  // The adapter of a row or task: the last that starts at or before it (one without rows starts where the next does).
  auto owner = [&](const int32_t* firsts, int at) -> int {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (firsts[mid] <= at ? lo : hi) = mid;
    }
    return lo;
  };
  for (int i = tid; i < none0 / kAdapterRowAlign; i += kGroupThreads)
    granules[i] = owner(first_row, i * kAdapterRowAlign);
  for (int i = tid; i < adapter_tasks; i += kGroupThreads) {
    const int a = owner(first_task, i);
    tasks[i] = make_int4(a, first_row[a] + (i - first_task[a]) * kAdapterTaskRows, first_row[a + 1], 0);
  }
  for (int a = warp; a < n; a += kGroupWarps) {  // padding rows, fewer than 32 an adapter
    const int i = last_row[a] + lane;
    if (i < first_row[a + 1]) order[i] = T;
  }
  if (tid == 0) {
    steps[0] = used;
    steps[1] = adapter_tasks + none_tasks;
    offsets[n] = none0;
    offsets[n + 1] = used;
  }
  for (int i = none0 / kAdapterRowAlign + tid; i < rows_cap / kAdapterRowAlign; i += kGroupThreads) granules[i] = n;
  for (int i = tid; i < none_tasks; i += kGroupThreads)
    tasks[adapter_tasks + i] = make_int4(n, none0 + i * kAdapterTaskRows, used, 0);
  for (int i = used + tid; i < rows_cap; i += kGroupThreads) order[i] = T;
  for (int tb = t0; tb < t1; tb += 32 * kAhead) {
    load(tb);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int a = ad[i];
      const uint32_t same = __match_any_sync(kFull, a);
      const int rank = __popc(same & ((1u << lane) - 1));
      const int base = a >= 0 ? mine[a] : 0;
      __syncwarp();
      if (a >= 0) {
        order[(a == n ? none0 : 0) + base + rank] = tb + 32 * i + lane;
        if (rank == 0) mine[a] = base + __popc(same);
      }
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_adapter_group(const int32_t* ids, int T, int n, int32_t* order, int32_t* offsets, int32_t* steps,
                                 cudaStream_t stream) {
  const int smem = kGroupWarps * (n + 1) * 4;
  // the same limit in every call: calls of several host threads may meet here
  const cudaError_t err = cudaFuncSetAttribute(adapter_group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kGroupWarps * (E4B_MAX_ADAPTERS + 1) * 4);
  if (err != cudaSuccess) return err;
  LaunchScope scope("adapter_group", stream);
  return launch_following(adapter_group_kernel, 1, kGroupThreads, smem, 0, stream, ids, T, n,
                          (int)adapter_rows_cap(T, n), order, offsets, steps);
}

}  // namespace e4b
