// Adapters of many requests beside a shared NF4 projection: the grouping of
// the tokens by adapter, and the projection's kernels.
//
//   y[t] = W x[t] + B[a] p[t],  p[t] = s[a] A[a] x[t]
#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ----------------------------------------------------------------------------
// Grouping: a stable counting sort of the tokens by adapter in one block.
// Every warp owns a contiguous run of tokens and a histogram row of its own in
// shared memory; lanes with equal ids find one another with a warp match, so
// that there are no shared-memory atomics and the order is fixed.  Two passes
// over the ids (count, place) around one scan over the adapters.
// ----------------------------------------------------------------------------
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;

__global__ void __launch_bounds__(kGroupThreads, 1)
    adapter_group_kernel(const int32_t* __restrict__ ids, int T, int n, int rows_cap, int32_t* __restrict__ order,
                         int32_t* __restrict__ offsets, int32_t* __restrict__ steps) {
  extern __shared__ int32_t table[];  // [kGroupWarps][n + 1]
  __shared__ int32_t wsum[3][kGroupWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cols = n + 1;
  for (int i = tid; i < kGroupWarps * cols; i += kGroupThreads) table[i] = 0;
  __syncthreads();
  const int per = ((T + kGroupWarps - 1) / kGroupWarps + 31) / 32 * 32;
  const int t0 = min(T, warp * per), t1 = min(T, t0 + per);
  int32_t* mine = table + warp * cols;
  auto adapter_of = [&](int t) -> int {
    const uint32_t a = (uint32_t)__ldg(ids + t);
    return a < (uint32_t)n ? (int)a : n;
  };
  int next = t0 + lane < t1 ? adapter_of(t0 + lane) : -1;
  for (int tb = t0; tb < t1; tb += 32) {
    const int a = next;
    if (tb + 32 + lane < t1)
      next = adapter_of(tb + 32 + lane);
    else
      next = -1;
    const uint32_t same = __match_any_sync(kFull, a);
    if (a >= 0 && (same & ((1u << lane) - 1)) == 0) mine[a] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Scan over the adapters (thread a owns adapter a): rows padded to 16, the
  // 256-row units its rows meet, and its 128-row projection tasks.
  int count = 0;
  if (tid < n)
    for (int w = 0; w < kGroupWarps; ++w) count += table[w * cols + tid];
  const int padded = (count + 15) / 16 * 16;
  auto block_scan = [&](int v, int which) -> int {  // exclusive prefix over the block
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[which][warp] = x;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += wsum[which][w];
    return base + x - v;
  };
  auto block_total = [&](int which) -> int {
    int s = 0;
    for (int w = 0; w < kGroupWarps; ++w) s += wsum[which][w];
    return s;
  };
  const int start = block_scan(padded, 0), end = start + padded;
  const int u0 = start / kAdapterUnitRows, u1 = padded ? (end - 1) / kAdapterUnitRows : u0 - 1;
  const int entry0 = block_scan(u1 - u0 + 1, 1);
  const int ntask = (padded + kAdapterTaskRows - 1) / kAdapterTaskRows;
  const int task0 = block_scan(ntask, 2);
  const int none0 = block_total(0), entries = block_total(1), adapter_tasks = block_total(2);
  int nnone = 0;
  for (int w = 0; w < kGroupWarps; ++w) nnone += table[w * cols + n];
  const int none_tasks = (nnone + kAdapterTaskRows - 1) / kAdapterTaskRows;
  const int used = none0 + nnone;
  const int units = (used + kAdapterUnitRows - 1) / kAdapterUnitRows;
  const AdapterSteps lay = adapter_steps_layout(rows_cap, n);
  int32_t* unit_start = steps + lay.unit_start;
  for (int u = tid; u <= rows_cap / kAdapterUnitRows; u += kGroupThreads) unit_start[u] = entries;
  __syncthreads();
  if (tid < n) {
    offsets[tid] = start;
    for (int u = u0; u <= u1; ++u) {
      const int i = entry0 + u - u0;
      int32_t* en = steps + lay.entries + 4 * i;
      en[0] = tid;
      en[1] = u;
      en[2] = start;
      en[3] = end;
      if (start <= u * kAdapterUnitRows) unit_start[u] = i;  // the first adapter with rows in unit u
    }
    for (int i = 0; i < ntask; ++i) {
      int32_t* tk = steps + lay.tasks + 4 * (task0 + i);
      tk[0] = tid;
      tk[1] = start + i * kAdapterTaskRows;
      tk[2] = end;
      tk[3] = 0;
    }
    for (int i = start + count; i < end; ++i) order[i] = T;  // padding rows
    // where each warp's tokens of this adapter start
    int at = start;
    for (int w = 0; w < kGroupWarps; ++w) {
      const int c = table[w * cols + tid];
      table[w * cols + tid] = at;
      at += c;
    }
  }
  if (tid == 0) {
    steps[0] = units;
    steps[1] = used;
    steps[2] = entries;
    steps[3] = adapter_tasks + none_tasks;
    int32_t* en = steps + lay.entries + 4 * entries;  // sentinel
    en[0] = -1;
    en[1] = -1;
    en[2] = en[3] = 0;
    offsets[n] = none0;
    offsets[n + 1] = used;
    int at = none0;
    for (int w = 0; w < kGroupWarps; ++w) {
      const int c = table[w * cols + n];
      table[w * cols + n] = at;
      at += c;
    }
  }
  for (int i = tid; i < none_tasks; i += kGroupThreads) {
    int32_t* tk = steps + lay.tasks + 4 * (adapter_tasks + i);
    tk[0] = n;
    tk[1] = none0 + i * kAdapterTaskRows;
    tk[2] = used;
    tk[3] = 0;
  }
  for (int i = used + tid; i < rows_cap; i += kGroupThreads) order[i] = T;
  __syncthreads();
  next = t0 + lane < t1 ? adapter_of(t0 + lane) : -1;
  for (int tb = t0; tb < t1; tb += 32) {
    const int a = next;
    if (tb + 32 + lane < t1)
      next = adapter_of(tb + 32 + lane);
    else
      next = -1;
    const uint32_t same = __match_any_sync(kFull, a);
    const int before = __popc(same & ((1u << lane) - 1));
    const int base = a >= 0 ? mine[a] : 0;
    __syncwarp();
    if (a >= 0) {
      order[base + before] = tb + lane;
      if (before == 0) mine[a] = base + __popc(same);
    }
    __syncwarp();
  }
}

}  // namespace

cudaError_t launch_adapter_group(const int32_t* ids, int T, int n, int32_t* order, int32_t* offsets, int32_t* steps,
                                 cudaStream_t stream) {
  const int smem = kGroupWarps * (n + 1) * 4;
  const cudaError_t err =
      cudaFuncSetAttribute(adapter_group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  LaunchScope scope("adapter_group", stream);
  adapter_group_kernel<<<1, kGroupThreads, smem, stream>>>(ids, T, n, (int)adapter_rows_cap(T, n), order, offsets,
                                                           steps);
  return cudaGetLastError();
}

}  // namespace e4b
