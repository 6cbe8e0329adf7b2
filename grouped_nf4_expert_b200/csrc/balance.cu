// The router's balance loss with its per-expert counts, and its gradient.
//
//   p[t,e] = exp(l[t,e] - lse[t]),  P[s,e] = sum_t p[t,e] / n_s,  f[s,e] = E counts[s,e] / (k n_s)
//   loss   = c_b mean_s sum_e f P + c_z mean_t lse^2
//   d l[t,j] = p[t,j] (c_b / (S' n_s) (f[s,j] - sum_e p[t,e] f[s,e]) + 2 c_z lse[t] / n)
//
// S' sequences and n tokens are the ones that take part.  Forward: one pass
// over the logits (maximum, sum of exponentials and probabilities of a row
// from one set of registers), the probabilities of a token range summed per
// expert in registers, one partial record per (range, sequence) piece; then
// one launch that joins a sequence's records in range order (so the sums do
// not depend on which block ran first) and, in its last block, the loss.
// Backward: one pass over the logits with lse given.
//
// What bounds them: HBM reads of the logits (forward) and reads plus writes
// of T x E float32 (backward); for small batches the two launches' latency.
// A group of G lanes owns a token, each lane four or more neighbouring
// columns (16-byte loads), G the smallest power of two with 4 G >= E, so that
// no lane idles at few experts and a row needs log2(G) shuffles.
#include <math.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 32;  // experts of one block of the joining launch

// First sequence whose end lies beyond token t (S: none); ends ascending.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int t) {
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// The columns of lane g of a group: 4 (v G + g) + 0..3 for v < V.  Rows start
// 16-byte aligned only when E is a multiple of 4; columns past E read as -inf.
template <int G, int V, bool ALIGNED>
__device__ __forceinline__ void load_row(const float* row, int g, int E, bool live, float (&l)[4 * V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 4 * (v * G + g);
    if (ALIGNED) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (live && c < E) q = __ldg(reinterpret_cast<const float4*>(row + c));
      l[4 * v] = q.x;
      l[4 * v + 1] = q.y;
      l[4 * v + 2] = q.z;
      l[4 * v + 3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) l[4 * v + i] = (live && c + i < E) ? __ldg(row + c + i) : -INFINITY;
    }
  }
}

struct FwdParams {
  const float* logits;
  const int32_t* ids;
  const int32_t* offsets;  // [S + 1] or nullptr
  const uint8_t* mask;     // [T] or nullptr
  float* lse;
  float* part_p;      // [slots, E] partial probability sums
  int32_t* part_c;    // [slots, E] partial counts
  float* part_z;      // [slots]
  int32_t* part_n;    // [slots] tokens
  int32_t* ticket;
  int T, E, k, S, per_block;
};

// Block b owns tokens [b C, (b + 1) C); every sequence that meets the range
// gives one piece, recorded in slot b + s (distinct along the staircase of
// pieces, which moves right in b or s at every step).
template <int G, int V, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(const FwdParams p) {
  extern __shared__ uint8_t smem[];
  float* sp = reinterpret_cast<float*>(smem);                  // [kWarps][E]
  int32_t* sc = reinterpret_cast<int32_t*>(sp + kWarps * p.E);  // [E]
  float* sz = reinterpret_cast<float*>(sc + p.E);               // [kWarps]
  int32_t* sn = reinterpret_cast<int32_t*>(sz + kWarps);        // [kWarps]
  constexpr int kTok = 32 / G;  // tokens of a warp at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G, sub = lane / G;
  const int E = p.E;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
  const int64_t r0 = (int64_t)blockIdx.x * p.per_block;
  const int t_end = (int)min((int64_t)p.T, r0 + p.per_block);
  int t0 = (int)min((int64_t)p.T, r0);
  int s = p.offsets ? sequence_of(p.offsets, p.S, t0) : 0;
  // tokens outside every sequence: lse = 0 like masked ones
  while (t0 < t_end) {
    int lo = 0, hi = p.T;
    if (p.offsets) {
      if (s >= p.S) {
        lo = hi = t_end;
      } else {
        lo = min(max(__ldg(p.offsets + s), t0), t_end);
        hi = min(max(__ldg(p.offsets + s + 1), lo), t_end);
      }
    }
    lo = max(lo, t0);
    hi = min(hi, t_end);
    for (int t = t0 + threadIdx.x; t < lo; t += kThreads) p.lse[t] = 0.0f;
    if (hi <= lo) {  // nothing of sequence s here
      t0 = lo;
      ++s;
      continue;
    }
    for (int e = threadIdx.x; e < E; e += kThreads) sc[e] = 0;
    float acc[4 * V];
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) acc[i] = 0.0f;
    float zsum = 0.0f;
    int n = 0;
    for (int tb = lo + warp * kTok; tb < hi; tb += kWarps * kTok) {
      const int t = tb + sub;
      const bool in = t < hi;
      const bool live = in && (p.mask == nullptr || __ldg(p.mask + t) != 0);
      float l[4 * V];
      load_row<G, V, ALIGNED>(p.logits + (size_t)(in ? t : lo) * E, g, E, live, l);
      float m = l[0];
#pragma unroll
      for (int i = 1; i < 4 * V; ++i) m = fmaxf(m, l[i]);
      m = group_max<G>(m);
      // a row of -inf alone (a masked token too) has no probabilities
      const float ms = (m == -INFINITY) ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        l[i] = expf(l[i] - ms);
        sum += l[i];
      }
      sum = group_sum<G>(sum);
      const float inv = (sum == 0.0f) ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) acc[i] = fmaf(l[i], inv, acc[i]);
      if (g == 0 && in) {
        const float lse = (sum == 0.0f) ? (live ? -INFINITY : 0.0f) : ms + logf(sum);
        p.lse[t] = lse;
        if (live) {
          if (sum != 0.0f) zsum = fmaf(lse, lse, zsum);
          ++n;
        }
      }
    }
    // this warp's tokens of one column: over the groups of the warp, then the warps in order
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) {
#pragma unroll
      for (int o = G; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], o);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      zsum += __shfl_xor_sync(kFull, zsum, o);
      n += __shfl_xor_sync(kFull, n, o);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        const int c = 4 * ((i >> 2) * G + g) + (i & 3);
        if (c < E) sp[warp * E + c] = acc[i];
      }
    }
    if (lane == 0) {
      sz[warp] = zsum;
      sn[warp] = n;
    }
    __syncthreads();
    // counts of the piece's slots (integer sums: any order)
    for (int64_t i = (int64_t)lo * p.k + threadIdx.x; i < (int64_t)hi * p.k; i += kThreads) {
      const uint32_t e = (uint32_t)__ldg(p.ids + i);
      if (e < (uint32_t)E && (p.mask == nullptr || __ldg(p.mask + (int)(i / p.k)) != 0)) atomicAdd(&sc[e], 1);
    }
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sp[w * E + e];
      p.part_p[slot * E + e] = v;
      p.part_c[slot * E + e] = sc[e];
    }
    if (threadIdx.x == 0) {
      float z = 0.0f;
      int c = 0;
      for (int w = 0; w < kWarps; ++w) {
        z += sz[w];
        c += sn[w];
      }
      p.part_z[slot] = z;
      p.part_n[slot] = c;
    }
    __syncthreads();  // the shared sums are read before the next piece
    t0 = hi;
    ++s;
  }
}

struct JoinParams {
  const int32_t* offsets;
  const float* part_p;
  const int32_t* part_c;
  const float* part_z;
  const int32_t* part_n;
  float* seq_dot;    // [S, slices] sum over a slice's experts of counts * probability sums
  float* seq_z;      // [S]
  int32_t* ticket;
  int32_t* counts;
  float* prob_sum;
  int32_t* tokens;
  float* loss;
  int T, E, k, S, per_block, slices;
  float c_b, c_z;
};

// Block (s, slice): the records of sequence s in range order, one expert a
// lane and every eighth record a warp.  The last block to finish adds up the
// loss, in sequence order.
__global__ void __launch_bounds__(kThreads) balance_join_kernel(const JoinParams p) {
  __shared__ float sp[kWarps][kSlice];
  __shared__ int32_t sc[kWarps][kSlice];
  __shared__ float red_a[kWarps], red_b[kWarps];
  __shared__ int red_n[kWarps], red_s[kWarps];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.x / p.slices, slice = blockIdx.x % p.slices;
  const int e = slice * kSlice + lane;
  int lo = p.offsets ? __ldg(p.offsets + s) : 0, hi = p.offsets ? __ldg(p.offsets + s + 1) : p.T;
  lo = min(max(lo, 0), p.T);
  hi = min(max(hi, lo), p.T);
  float a = 0.0f, z = 0.0f;
  int c = 0, n = 0;
  if (hi > lo) {
    const int b0 = lo / p.per_block, b1 = (hi - 1) / p.per_block;
    for (int b = b0 + warp; b <= b1; b += kWarps) {
      const size_t slot = (size_t)b + s;
      if (e < p.E) {
        a += p.part_p[slot * p.E + e];
        c += p.part_c[slot * p.E + e];
      }
    }
    if (warp == 0) {
      for (int b = b0 + lane; b <= b1; b += 32) {
        z += p.part_z[(size_t)b + s];
        n += p.part_n[(size_t)b + s];
      }
    }
  }
  sp[warp][lane] = a;
  sc[warp][lane] = c;
  __syncthreads();
  if (warp == 0) {
    a = 0.0f;
    c = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a += sp[w][lane];
      c += sc[w][lane];
    }
    if (e < p.E) {
      p.counts[(size_t)s * p.E + e] = c;
      p.prob_sum[(size_t)s * p.E + e] = a;
    }
    float dot = (e < p.E) ? (float)c * a : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      dot += __shfl_xor_sync(kFull, dot, o);
      z += __shfl_xor_sync(kFull, z, o);
      n += __shfl_xor_sync(kFull, n, o);
    }
    if (lane == 0) {
      p.seq_dot[(size_t)s * p.slices + slice] = dot;
      if (slice == 0) {
        p.seq_z[s] = z;
        p.tokens[s] = n;
      }
      __threadfence();
      last = atomicAdd(p.ticket, 1) == (int)gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // balance = (1 / S') sum_s (E / (k n_s^2)) sum_e counts psum;  z = sum_s seq_z / n
  float bal = 0.0f, zz = 0.0f;
  int nt = 0, ns = 0;
  for (int q = threadIdx.x; q < p.S; q += kThreads) {
    const int m = __ldcg(p.tokens + q);
    if (m > 0) {
      float d = 0.0f;
      for (int i = 0; i < p.slices; ++i) d += __ldcg(p.seq_dot + (size_t)q * p.slices + i);
      bal += d * ((float)p.E / ((float)p.k * (float)m)) / (float)m;
      zz += __ldcg(p.seq_z + q);
      nt += m;
      ++ns;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    bal += __shfl_xor_sync(kFull, bal, o);
    zz += __shfl_xor_sync(kFull, zz, o);
    nt += __shfl_xor_sync(kFull, nt, o);
    ns += __shfl_xor_sync(kFull, ns, o);
  }
  if (lane == 0) {
    red_a[warp] = bal;
    red_b[warp] = zz;
    red_n[warp] = nt;
    red_s[warp] = ns;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    bal = zz = 0.0f;
    nt = ns = 0;
    for (int w = 0; w < kWarps; ++w) {
      bal += red_a[w];
      zz += red_b[w];
      nt += red_n[w];
      ns += red_s[w];
    }
    bal = ns > 0 ? bal / (float)ns : 0.0f;
    zz = nt > 0 ? zz / (float)nt : 0.0f;
    p.tokens[p.S] = nt;
    p.tokens[p.S + 1] = ns;
    p.loss[0] = p.c_b * bal + p.c_z * zz;
    p.loss[1] = bal;
    p.loss[2] = zz;
  }
}

struct BwdParams {
  const float* logits;
  const int32_t* offsets;
  const uint8_t* mask;
  const int32_t* counts;
  const int32_t* tokens;
  const float* lse;
  const float* dloss;
  float* d_logits;
  int T, E, k, S, per_warp, accumulate;
  float c_b, c_z;
};

// A warp owns a run of tokens; the f of the sequence at hand stays in
// registers and is read again where the sequence changes.
template <int G, int V, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BwdParams p) {
  constexpr int kTok = 32 / G;
  const int lane = threadIdx.x & 31, g = lane % G, sub = lane / G;
  const int64_t w0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.per_warp;
  if (w0 >= p.T) return;
  const int t_end = (int)min((int64_t)p.T, w0 + p.per_warp);
  const int E = p.E;
  const float up = p.dloss ? __ldg(p.dloss) : 1.0f;
  const int n_tok = __ldg(p.tokens + p.S), n_seq = __ldg(p.tokens + p.S + 1);
  const float zc = n_tok > 0 ? up * 2.0f * p.c_z / (float)n_tok : 0.0f;
  int t0 = (int)w0;
  int s = p.offsets ? sequence_of(p.offsets, p.S, t0) : 0;
  while (t0 < t_end) {
    // [t0, hi): tokens of sequence s, or (s == S, or before its start) of none
    bool inside = true;
    int hi = t_end;
    if (p.offsets) {
      if (s >= p.S) {
        inside = false;
      } else {
        const int a = __ldg(p.offsets + s), b = __ldg(p.offsets + s + 1);
        if (t0 < a) {
          inside = false;
          hi = min(a, t_end);
        } else {
          hi = min(max(b, t0), t_end);
          if (hi <= t0) {
            ++s;
            continue;
          }
        }
      }
    }
    float f[4 * V];
    float bc = 0.0f;
    if (inside) {
      const int n_s = __ldg(p.tokens + s);
      const float fc = n_s > 0 ? (float)E / ((float)p.k * (float)n_s) : 0.0f;
      bc = n_s > 0 ? up * p.c_b / ((float)n_seq * (float)n_s) : 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        const int c = 4 * ((i >> 2) * G + g) + (i & 3);
        f[i] = c < E ? fc * (float)__ldg(p.counts + (size_t)s * E + c) : 0.0f;
      }
    }
    for (int tb = t0; tb < hi; tb += kTok) {
      const int t = tb + sub;
      const bool in = t < hi;
      const bool live = in && inside && (p.mask == nullptr || __ldg(p.mask + t) != 0);
      float l[4 * V];
      load_row<G, V, ALIGNED>(p.logits + (size_t)(in ? t : t0) * E, g, E, live, l);
      const float lse = live ? __ldg(p.lse + t) : 0.0f;
      const bool some = lse != -INFINITY;  // a row of -inf alone has no probabilities
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        l[i] = some ? expf(l[i] - lse) : 0.0f;
        dot = fmaf(l[i], live ? f[i] : 0.0f, dot);
      }
      dot = group_sum<G>(dot);
      const float zt = some ? zc * lse : 0.0f;
      if (in) {
        float* row = p.d_logits + (size_t)t * E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = 4 * (v * G + g);
          float d[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = live ? l[4 * v + i] * fmaf(bc, f[4 * v + i] - dot, zt) : 0.0f;
          if (ALIGNED) {
            if (c < E) {
              float4* q = reinterpret_cast<float4*>(row + c);
              float4 o = make_float4(d[0], d[1], d[2], d[3]);
              if (p.accumulate) {
                if (!live) continue;
                const float4 w = *q;
                o = make_float4(w.x + d[0], w.y + d[1], w.z + d[2], w.w + d[3]);
              }
              *q = o;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < E) {
                if (!p.accumulate)
                  row[c + i] = d[i];
                else if (live)
                  row[c + i] += d[i];
              }
          }
        }
      }
    }
    t0 = hi;
  }
}

// Runs F<G, V, ALIGNED> for E columns.
template <template <int, int, bool> class F, typename... Args>
cudaError_t dispatch_columns(int E, Args... args) {
  const bool al = (E & 3) == 0;
#define E4B_BAL(G, V) return al ? F<G, V, true>::run(args...) : F<G, V, false>::run(args...)
  if (E <= 4) E4B_BAL(1, 1);
  if (E <= 8) E4B_BAL(2, 1);
  if (E <= 16) E4B_BAL(4, 1);
  if (E <= 32) E4B_BAL(8, 1);
  if (E <= 64) E4B_BAL(16, 1);
  if (E <= 128) E4B_BAL(32, 1);
  if (E <= 256) E4B_BAL(32, 2);
  if (E <= 512) E4B_BAL(32, 4);
  E4B_BAL(32, 8);
#undef E4B_BAL
}

template <int G, int V, bool ALIGNED>
struct RunFwd {
  static cudaError_t run(FwdParams p, int grid, cudaStream_t stream) {
    const int smem = (kWarps * p.E + p.E + 2 * kWarps) * 4;
    balance_fwd_kernel<G, V, ALIGNED><<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  }
};
template <int G, int V, bool ALIGNED>
struct RunBwd {
  static cudaError_t run(BwdParams p, int grid, cudaStream_t stream) {
    balance_bwd_kernel<G, V, ALIGNED><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
};

constexpr int kMaxBlocks = 2 * 148;

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
int balance_blocks(int T) {
  // at least a token for every warp of a block, at most kMaxBlocks ranges
  const int b = (T + kWarps - 1) / kWarps;
  return b < 1 ? 1 : (b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) {
  const size_t slots = (size_t)balance_blocks(T) + S;
  const size_t slices = (E + kSlice - 1) / kSlice;
  return 256 + 2 * align256(slots * E * 4) + 2 * align256(slots * 4) + align256((size_t)S * slices * 4) +
         align256((size_t)S * 4);
}

cudaError_t launch_balance_fwd(const BalanceHost& h, void* ws, cudaStream_t stream) {
  const int want = balance_blocks(h.T);
  const int per = (h.T + want - 1) / want;
  const int grid = (h.T + per - 1) / per;
  const size_t slots = (size_t)want + h.S;
  const int slices = (h.E + kSlice - 1) / kSlice;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* at = w;
    w += align256(bytes);
    return at;
  };
  FwdParams p;
  p.ticket = reinterpret_cast<int32_t*>(take(256));
  p.part_p = reinterpret_cast<float*>(take(slots * h.E * 4));
  p.part_c = reinterpret_cast<int32_t*>(take(slots * h.E * 4));
  p.part_z = reinterpret_cast<float*>(take(slots * 4));
  p.part_n = reinterpret_cast<int32_t*>(take(slots * 4));
  JoinParams j;
  j.seq_dot = reinterpret_cast<float*>(take((size_t)h.S * slices * 4));
  j.seq_z = reinterpret_cast<float*>(take((size_t)h.S * 4));
  p.logits = h.logits;
  p.ids = h.ids;
  p.offsets = h.offsets;
  p.mask = h.mask;
  p.lse = h.lse;
  p.T = h.T;
  p.E = h.E;
  p.k = h.k;
  p.S = h.S;
  p.per_block = per;
  {
    LaunchScope scope("balance_fwd", stream);
    const cudaError_t err = dispatch_columns<RunFwd>(h.E, p, grid, stream);
    if (err != cudaSuccess) return err;
  }
  j.offsets = h.offsets;
  j.part_p = p.part_p;
  j.part_c = p.part_c;
  j.part_z = p.part_z;
  j.part_n = p.part_n;
  j.ticket = p.ticket;
  j.counts = h.counts;
  j.prob_sum = h.prob_sum;
  j.tokens = h.tokens;
  j.loss = h.loss;
  j.T = h.T;
  j.E = h.E;
  j.k = h.k;
  j.S = h.S;
  j.per_block = per;
  j.slices = slices;
  j.c_b = h.c_b;
  j.c_z = h.c_z;
  LaunchScope scope("balance_join", stream);
  balance_join_kernel<<<h.S * slices, kThreads, 0, stream>>>(j);
  return cudaGetLastError();
}

cudaError_t launch_balance_bwd(const BalanceHost& h, const float* dloss, bool accumulate, float* d_logits,
                               int num_sms, cudaStream_t stream) {
  BwdParams p;
  p.logits = h.logits;
  p.offsets = h.offsets;
  p.mask = h.mask;
  p.counts = h.counts;
  p.tokens = h.tokens;
  p.lse = h.lse;
  p.dloss = dloss;
  p.d_logits = d_logits;
  p.T = h.T;
  p.E = h.E;
  p.k = h.k;
  p.S = h.S;
  p.accumulate = accumulate ? 1 : 0;
  p.c_b = h.c_b;
  p.c_z = h.c_z;
  // runs of tokens: every warp of eight blocks an SM takes one
  const int64_t warps = (int64_t)num_sms * 8 * kWarps;
  p.per_warp = (int)((h.T + warps - 1) / warps);
  const int64_t used = ((int64_t)h.T + p.per_warp - 1) / p.per_warp;
  const int grid = (int)((used + kWarps - 1) / kWarps);
  LaunchScope scope("balance_bwd", stream);
  return dispatch_columns<RunBwd>(h.E, p, grid, stream);
}

}  // namespace e4b
