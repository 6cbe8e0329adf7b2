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
  const int none0 = block_total(0), entries = block_total(1), tasks = block_total(2);
  int nnone = 0;
  for (int w = 0; w < kGroupWarps; ++w) nnone += table[w * cols + n];
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
    steps[3] = tasks;
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

// ----------------------------------------------------------------------------
// Plain kernels
// ----------------------------------------------------------------------------
__device__ __forceinline__ float bf(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t to_bf(float f) {
  const __nv_bfloat16 b = __float2bfloat16_rn(f);
  return *reinterpret_cast<const uint16_t*>(&b);
}
__device__ __forceinline__ int adapter_of_row(const int32_t* offsets, int n, int row) {
  int lo = 0, hi = n;  // the last group whose start is <= row (empty groups share a start with the next)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= row)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// out[row, j] = bf16(s sum_k src[t, k] F[a](k, j)): F = A[a][j][k], or B[a][k][j] with MN
template <bool MN>
__global__ void adapter_rows_kernel(const uint16_t* src, const uint16_t* fac, const float* scale,
                                    const int32_t* order, const int32_t* offsets, int T, int K, int n, int r,
                                    uint16_t* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int used = offsets[n];
  for (int row = blockIdx.x; row < used; row += gridDim.x) {
    const int a = adapter_of_row(offsets, n, row), t = order[row];
    for (int j = warp; j < r; j += blockDim.x / 32) {
      float acc = 0.0f;
      if (t < T)
        for (int k = lane; k < K; k += 32) {
          const size_t i = MN ? ((size_t)a * K + k) * r + j : ((size_t)a * r + j) * K + k;
          acc = fmaf(bf(src[(size_t)t * K + k]), bf(fac[i]), acc);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFull, acc, o);
      if (lane == 0) out[(size_t)row * r + j] = to_bf(scale[a] * acc);
    }
  }
}

// 64 rows x 64 outputs a block: out[t, o] = sum_i src[t, i] W(o, i) + sum_j low[row, j] F[a](o, j)
template <bool MN>
__global__ void __launch_bounds__(256) adapter_gemm_kernel(const uint16_t* src, const uint8_t* nf4,
                                                           const float* absmax, const uint16_t* low,
                                                           const uint16_t* fac, const int32_t* order,
                                                           const int32_t* offsets, int T, int K, int N, int n, int r,
                                                           uint16_t* out) {
  __shared__ float xs[32][65], ws[32][65];
  __shared__ float lv[16];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int R = MN ? N : K, O = MN ? K : N;
  const int row0 = blockIdx.y * 64, o0 = blockIdx.x * 64;
  if (row0 >= offsets[n + 1]) return;
  if (tid < 16) lv[tid] = nf4_level(tid);
  float acc[4][4] = {};
  for (int i0 = 0; i0 < R; i0 += 32) {
    __syncthreads();
    for (int q = tid; q < 64 * 32; q += 256) {
      const int i = q & 31, m = q >> 5, t = order[row0 + m];
      xs[i][m] = (t < T && i0 + i < R) ? bf(src[(size_t)t * R + i0 + i]) : 0.0f;
      const int wi = MN ? (q >> 6) : i, wo = MN ? (q & 63) : m;
      const int nn = MN ? i0 + wi : o0 + wo, kk = MN ? o0 + wo : i0 + wi;
      float w = 0.0f;
      if (nn < N && kk < K) {
        const uint8_t b = nf4[(size_t)nn * (K / 2) + kk / 2];
        w = bf(to_bf(__fmul_rn(lv[(kk & 1) ? b & 15 : b >> 4], absmax[(size_t)nn * (K / 64) + kk / 64])));
      }
      ws[wi][wo] = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(xs[i][ty + 16 * u], ws[i][tx + 16 * v], acc[u][v]);
  }
  for (int u = 0; u < 4; ++u) {
    const int row = row0 + ty + 16 * u, t = order[row];
    if (t >= T) continue;
    const int a = adapter_of_row(offsets, n, row);
    for (int v = 0; v < 4; ++v) {
      const int o = o0 + tx + 16 * v;
      if (o >= O) continue;
      float d = acc[u][v];
      if (a < n)
        for (int j = 0; j < r; ++j) {
          const size_t i = MN ? ((size_t)a * r + j) * K + o : ((size_t)a * N + o) * r + j;
          d = fmaf(bf(low[(size_t)row * r + j]), bf(fac[i]), d);
        }
      out[(size_t)t * O + o] = to_bf(d);
    }
  }
}

// out[a] = sum over its rows of low^T act: [r, F] (transposed) or [F, r]
template <bool TR>
__global__ void __launch_bounds__(256) adapter_wgrad_kernel(const uint16_t* act, const uint16_t* low,
                                                            const int32_t* order, const int32_t* offsets, int T,
                                                            int F, int r, uint16_t* out) {
  const int a = blockIdx.y, f = blockIdx.x * 64 + (threadIdx.x & 63), jg = threadIdx.x >> 6;
  if (f >= F) return;
  float acc[16] = {};
  for (int row = offsets[a]; row < offsets[a + 1]; ++row) {
    const int t = order[row];
    if (t >= T) continue;
    const float v = bf(act[(size_t)t * F + f]);
    for (int i = 0; i < 16; ++i)
      if (jg + 4 * i < r) acc[i] = fmaf(v, bf(low[(size_t)row * r + jg + 4 * i]), acc[i]);
  }
  for (int i = 0; i < 16; ++i) {
    const int j = jg + 4 * i;
    if (j < r) out[TR ? ((size_t)a * r + j) * F + f : ((size_t)a * F + f) * r + j] = to_bf(acc[i]);
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

cudaError_t launch_adapter_rows(const AdapterProjHost& h, bool mn, const uint16_t* src, const uint16_t* fac,
                                uint16_t* out, cudaStream_t stream) {
  const int grid = (int)(h.rows_cap < 4096 ? h.rows_cap : 4096);
  LaunchScope scope(mn ? "adapter_rows_dy" : "adapter_rows_x", stream);
  if (mn)
    adapter_rows_kernel<true><<<grid, 256, 0, stream>>>(src, fac, h.scale, h.order, h.offsets, h.T, h.N, h.n, h.r, out);
  else
    adapter_rows_kernel<false><<<grid, 256, 0, stream>>>(src, fac, h.scale, h.order, h.offsets, h.T, h.K, h.n, h.r,
                                                         out);
  return cudaGetLastError();
}

cudaError_t launch_adapter_gemm(const AdapterProjHost& h, bool mn, const uint16_t* src, const uint16_t* low,
                                const uint16_t* fac, uint16_t* out, cudaStream_t stream) {
  const dim3 grid(((mn ? h.K : h.N) + 63) / 64, (unsigned)(h.rows_cap / 64));
  LaunchScope scope(mn ? "adapter_gemm_dgrad" : "adapter_gemm_fwd", stream);
  if (mn)
    adapter_gemm_kernel<true><<<grid, 256, 0, stream>>>(src, h.nf4, h.absmax, low, fac, h.order, h.offsets, h.T, h.K,
                                                        h.N, h.n, h.r, out);
  else
    adapter_gemm_kernel<false><<<grid, 256, 0, stream>>>(src, h.nf4, h.absmax, low, fac, h.order, h.offsets, h.T, h.K,
                                                         h.N, h.n, h.r, out);
  return cudaGetLastError();
}

cudaError_t launch_adapter_wgrad(const AdapterProjHost& h, const uint16_t* x, const uint16_t* dY, const uint16_t* p,
                                 const uint16_t* q, uint16_t* dA, uint16_t* dB, cudaStream_t stream) {
  LaunchScope scope("adapter_wgrad", stream);
  adapter_wgrad_kernel<true><<<dim3((h.K + 63) / 64, h.n), 256, 0, stream>>>(x, q, h.order, h.offsets, h.T, h.K, h.r,
                                                                             dA);
  adapter_wgrad_kernel<false><<<dim3((h.N + 63) / 64, h.n), 256, 0, stream>>>(dY, p, h.order, h.offsets, h.T, h.N, h.r,
                                                                              dB);
  return cudaGetLastError();
}

}  // namespace e4b
