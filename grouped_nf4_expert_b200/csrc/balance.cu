// The router's balance loss with its per-expert counts, and its gradient.
//
//   p[t,e] = exp(l[t,e] - lse[t]),  P[s,e] = sum_t p[t,e] / n_s,  f[s,e] = E counts[s,e] / (k n_s)
//   loss   = c_b mean_s sum_e f P + c_z mean_t lse^2
//   d l[t,j] = p[t,j] (c_b / (S' n_s) (f[s,j] - sum_e p[t,e] f[s,e]) + 2 c_z lse[t] / n)
//
// S' sequences and n tokens are the ones that take part.  Forward: one pass
// over the logits (maximum, sum of exponentials and probabilities of a row
// from one set of registers), the probabilities of a token range summed per
// expert in registers, one partial record per (range, sequence) piece; more
// blocks at the end of the grid wait for the records (a counter in the workspace,
// bounded wait; the blocks they wait for come first and never wait), add a
// sequence's records in range order, so that the sums do not depend on which
// block ran first, and the last of them adds up their shares of the loss.  A
// second launch in their place cost the host 4.5 us and the GPU 10 to 15.
// Backward: one pass over the logits with lse given, each row's probabilities divided by their sum.
//
// What bounds them: HBM reads of the logits (forward) and reads plus writes
// of T x E float32 (backward); for small batches the launch.  131072 tokens of
// 64 experts: backward 11.4 us with the logits in L2 (5.9 TB/s), 15 us from cold
// caches; forward 16 to 18.5 us, of which the pass over the logits takes 10 and the
// records, their counter and the join the rest.
// A group of G lanes owns a token, each lane 16 columns in runs of four
// (16-byte loads), G the smallest power of two with 16 G >= E: with four columns
// a lane the shuffles and the other work per token and lane were the limit, not
// memory (forward 46 us).
#include <math.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"
#include "launch.cuh"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 8;  // experts of a joining item: 8 lanes, so that 32 records are read at a time

// First sequence whose end lies beyond token t (S: none); ends ascending.  Whole warp: 32 ends a round trip, where
// a binary search would wait for memory log2(S) times.
__device__ __forceinline__ int sequence_of(const int32_t* offsets, int S, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = S;  // the answer lies in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const bool past = at < hi && __ldg(offsets + at + 1) <= t;  // sequence `at` ends at or before t
    const int n = __popc(__ballot_sync(kFull, past));
    if (n == 0) return lo;
    lo += (n - 1) * step + 1;
    hi = min(hi, lo + step - 1);
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

// exp(x) for x up to 0 (or a rounding above): the exponential of 2 of x log2(e), three operations a value where expf
// has about nine (131072 tokens of 64 experts, both directions, before the gradient's sums: expf 34.9 us, this
// 29.5 us).  Relative error (1.3 |x| + 4) 2^-24: the
// product's rounding and the constant's, and the instruction's.  -inf gives 0; probabilities below 2^-126 are 0.
__device__ __forceinline__ float exp_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// The columns of lane g of a group: 4 (v G + g) + 0..3 for v < V.  Rows start
// 16-byte aligned only when E is a multiple of 4; columns past E, and rows that
// are not there, read as -inf.
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
  DeviceError* err;   // the workspace's front: `ready` record blocks done, `left` joining blocks done
  float2* part;       // [slots, E] (probability sum, count as an int's bits)
  float2* part_zn;    // [slots] (sum of lse^2, tokens as an int's bits)
  float4* joined;     // [joining blocks] its items' balance, sum of lse^2, tokens and sequences as ints' bits
  int32_t* counts;
  float* prob_sum;
  int32_t* tokens;
  float* lse;
  float* loss;
  int T, E, k, S, per_block, slices, blocks, join_blocks;  // record blocks, then joining blocks
  float c_b, c_z;
};

__device__ __forceinline__ int2 sequence_range(const FwdParams& p, int s) {
  if (p.offsets == nullptr) return make_int2(0, p.T);
  const int lo = min(max(__ldg(p.offsets + s), 0), p.T);
  return make_int2(lo, min(max(__ldg(p.offsets + s + 1), lo), p.T));
}

// Balance terms, sums of lse^2, tokens and sequences with tokens.
struct Joined {
  float bal, z;
  int n, s;
};
__device__ __forceinline__ void add(Joined& a, const Joined& b) {
  a.bal += b.bal;
  a.z += b.z;
  a.n += b.n;
  a.s += b.s;
}

// The join: item (s, slice) adds the records of sequence s in range order: W warps take every W-th 4-record group, a
// lane one expert of every fourth record.  A block an item (W = 8) while there are blocks enough, else a warp.  A
// sequence's term of the balance is E / (k n_s^2) sum_e counts * probability sums.  Lane 0's result counts.
template <int W>
__device__ Joined join_items(const FwdParams& p, int first, int step, int2 range) {
  __shared__ float sp[kWarps][kSlice];
  __shared__ int32_t sc[kWarps][kSlice];
  __shared__ float sz[kWarps];
  __shared__ int32_t sn[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = lane & (kSlice - 1), row = lane / kSlice;
  const int part_of = W == 1 ? 0 : warp;
  Joined sum = {0.0f, 0.0f, 0, 0};
  for (int item = first; item < p.S * p.slices; item += step) {
    const int s = item / p.slices, slice = item - s * p.slices, e = slice * kSlice + col;
    if (item != first) range = sequence_range(p, s);
    const int lo = range.x, hi = range.y;
    const int b0 = lo / p.per_block, b1 = hi > lo ? (hi - 1) / p.per_block : b0 - 1;
    float a = 0.0f, z = 0.0f;
    int c = 0, n = 0;
    constexpr int kAhead = 8, kStep = W * 4;
#pragma unroll 2
    for (int b = b0 + 32 * part_of + lane; b <= b1; b += 32 * W) {
      const float2 v = __ldcg(p.part_zn + (size_t)b + s);
      z += v.x;
      n += __float_as_int(v.y);
    }
    for (int b = b0 + 4 * part_of + row; b <= b1; b += kStep * kAhead) {
      float2 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int at = b + i * kStep;
        v[i] = (at <= b1 && e < p.E) ? __ldcg(p.part + ((size_t)at + s) * p.E + e) : make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        a += v[i].x;
        c += __float_as_int(v[i].y);
      }
    }
#pragma unroll
    for (int o = kSlice; o < 32; o <<= 1) {
      a += __shfl_xor_sync(kFull, a, o);
      c += __shfl_xor_sync(kFull, c, o);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(kFull, z, o);
      n += __shfl_xor_sync(kFull, n, o);
    }
    if constexpr (W > 1) {
      if (row == 0) {
        sp[warp][col] = a;
        sc[warp][col] = c;
      }
      if (lane == 0) {
        sz[warp] = z;
        sn[warp] = n;
      }
      __syncthreads();
      a = z = 0.0f;
      c = n = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        a += sp[w][col];
        c += sc[w][col];
        z += sz[w];
        n += sn[w];
      }
    }
    if (part_of == 0) {
      if (row == 0 && e < p.E) {
        p.counts[(size_t)s * p.E + e] = c;
        p.prob_sum[(size_t)s * p.E + e] = a;
      }
      float dot = (row == 0 && e < p.E) ? (float)c * a : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      if (n > 0) sum.bal += dot * ((float)p.E / ((float)p.k * (float)n)) / (float)n;
      if (slice == 0) {
        if (lane == 0) p.tokens[s] = n;
        if (n > 0) {
          sum.z += z;
          sum.n += n;
          ++sum.s;
        }
      }
    }
    if constexpr (W > 1) __syncthreads();
  }
  return sum;
}

__device__ __forceinline__ void write_loss(const FwdParams& p, const Joined& v) {
  const float bal = v.s > 0 ? v.bal / (float)v.s : 0.0f;
  const float zz = v.n > 0 ? v.z / (float)v.n : 0.0f;
  p.tokens[p.S] = v.n;
  p.tokens[p.S + 1] = v.s;
  p.loss[0] = p.c_b * bal + p.c_z * zz;
  p.loss[1] = bal;
  p.loss[2] = zz;
}

__device__ __forceinline__ void empty_sequence(const FwdParams& p, int s) {
  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    p.counts[(size_t)s * p.E + e] = 0;
    p.prob_sum[(size_t)s * p.E + e] = 0.0f;
  }
  if (threadIdx.x == 0) p.tokens[s] = 0;
}

// A block behind the record blocks.
__device__ void join_block(const FwdParams& p) {
  __shared__ int flag;
  const int joiner = (int)blockIdx.x - p.blocks, items = p.S * p.slices;
  const bool wide = items <= p.join_blocks;
  const int first = wide ? joiner : joiner * kWarps + (threadIdx.x >> 5);
  int2 range = make_int2(0, 0);
  if (first < items) range = sequence_range(p, first / p.slices);
  if (threadIdx.x == 0) {
    const long long c0 = clock64(), limit = wait_limit_cycles(kDefaultTimeoutNs);
    int v;
    do {
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(&p.err->ready) : "memory");
    } while (v < p.blocks && clock64() - c0 < limit);
    flag = v >= p.blocks;
    if (!flag) record_error(p.err, E4B_ERR_DEVICE_TIMEOUT, 700);
  }
  __syncthreads();
  if (!flag) return;
  __shared__ Joined warps[kWarps];
  const Joined mine = wide ? join_items<kWarps>(p, first, p.join_blocks, range)
                           : join_items<1>(p, first, p.join_blocks * kWarps, range);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    Joined v = {0.0f, 0.0f, 0, 0};
    for (int w = 0; w < kWarps; ++w) add(v, warps[w]);
    p.joined[joiner] = make_float4(v.bal, v.z, __int_as_float(v.n), __int_as_float(v.s));
    __threadfence();
    flag = atomicAdd(&p.err->left, 1) == p.join_blocks - 1;
  }
  __syncthreads();
  if (!flag || threadIdx.x >= 32) return;
  __threadfence();
  Joined v = {0.0f, 0.0f, 0, 0};
  for (int b = threadIdx.x; b < p.join_blocks; b += 32) {
    const float4 q = __ldcg(p.joined + b);
    add(v, {q.x, q.y, __float_as_int(q.z), __float_as_int(q.w)});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add(v, {__shfl_xor_sync(kFull, v.bal, o), __shfl_xor_sync(kFull, v.z, o), __shfl_xor_sync(kFull, v.n, o),
            __shfl_xor_sync(kFull, v.s, o)});
  if (threadIdx.x == 0) {
    write_loss(p, v);
    p.err->ready = p.err->left = 0;
  }
}

// Resident blocks of the forward on an SM, so that one's loads meet another's arithmetic (131072 tokens of 64 experts:
// two 20.5 us, four 18.6 us).
constexpr int fwd_blocks(int V) { return V == 8 ? 2 : 4; }

// Block b owns tokens [b C, (b + 1) C); every sequence that meets the range
// gives one piece, recorded in slot b + s (distinct along the staircase of
// pieces, which moves right in b or s at every step).  ONE: a single block
// covers the batch; its pieces are the sequences and need no records.
template <int G, int V, bool ALIGNED, bool ONE>
__global__ void __launch_bounds__(kThreads, fwd_blocks(V)) balance_fwd_kernel(const FwdParams p) {
  grid_wait();
  grid_launch_dependents();
  if (!ONE && (int)blockIdx.x >= p.blocks) {
    join_block(p);
    return;
  }
  extern __shared__ uint8_t smem[];
  float* sp = reinterpret_cast<float*>(smem);                  // [kWarps][E]
  int32_t* sc = reinterpret_cast<int32_t*>(sp + kWarps * p.E);  // [E]
  float* sz = reinterpret_cast<float*>(sc + p.E);               // [kWarps]
  int32_t* sn = reinterpret_cast<int32_t*>(sz + kWarps);        // [kWarps]
  constexpr int kTok = 32 / G;  // tokens of a warp at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % G, sub = lane / G;
  const int E = p.E;
  const bool few_ids = p.k <= 2 * G;
  const int64_t r0 = (int64_t)blockIdx.x * p.per_block;
  const int t_end = (int)min((int64_t)p.T, r0 + p.per_block);
  int t0 = (int)min((int64_t)p.T, r0);
  int s = p.offsets && !ONE ? sequence_of(p.offsets, p.S, t0) : 0;
  Joined total = {0.0f, 0.0f, 0, 0};  // (ONE, thread 0) the sequences so far
  while (t0 < t_end) {
    int lo = t0, hi = t_end;
    if (p.offsets) {
      if (s >= p.S) {
        lo = hi = t_end;
      } else {
        lo = min(max(__ldg(p.offsets + s), t0), t_end);
        hi = min(max(__ldg(p.offsets + s + 1), lo), t_end);
      }
    }
    for (int t = t0 + threadIdx.x; t < lo; t += kThreads) p.lse[t] = 0.0f;  // tokens of no sequence
    if (hi <= lo) {  // nothing of sequence s here
      if (ONE && s < p.S) empty_sequence(p, s);
      t0 = lo;
      ++s;
      continue;
    }
    for (int e = threadIdx.x; e < E; e += kThreads) sc[e] = 0;
    __syncthreads();
    float acc[4 * V];
#pragma unroll
    for (int i = 0; i < 4 * V; ++i) acc[i] = 0.0f;
    float zsum = 0.0f;
    int n = 0;
    for (int t = lo + warp * kTok + sub; t - sub < hi; t += kWarps * kTok) {
      float l[4 * V];
      int id[2];
      const bool in = t < hi;
      load_row<G, V, ALIGNED>(p.logits + (size_t)(in ? t : lo) * E, g, E, in, l);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        id[j] = in && few_ids && g + j * G < p.k ? __ldg(p.ids + (size_t)t * p.k + g + j * G) : -1;
      const bool live = in && (p.mask == nullptr || __ldg(p.mask + t) != 0);
      if (!live) {  // a masked token's values are not looked at
#pragma unroll
        for (int i = 0; i < 4 * V; ++i) l[i] = -INFINITY;
        id[0] = id[1] = -1;
      }
      float m = l[0];
#pragma unroll
      for (int i = 1; i < 4 * V; ++i) m = fmaxf(m, l[i]);
      m = group_max<G>(m);
      // a row of -inf alone (a masked token too) has no probabilities
      const float ms = (m == -INFINITY) ? 0.0f : m;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        l[i] = exp_of(l[i] - ms);
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
      // the token's slots (integer sums: any order)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if ((uint32_t)id[j] < (uint32_t)E) atomicAdd(&sc[id[j]], 1);
    }
    if (!few_ids) {  // more slots than two a lane: the piece's ids in a pass of their own
      const uint32_t n_ids = (uint32_t)(hi - lo) * p.k;
      const int32_t* at = p.ids + (size_t)lo * p.k;
      constexpr int kAhead = 8;
      for (uint32_t i0 = threadIdx.x; i0 < n_ids; i0 += kThreads * kAhead) {
        uint32_t e[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const uint32_t i = i0 + j * kThreads;
          e[j] = i < n_ids ? (uint32_t)__ldg(at + i) : kFull;
        }
        if (p.mask != nullptr) {  // loads of their own, all eight in flight
          uint8_t on[kAhead];
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            on[j] = __ldg(p.mask + lo + min(i0 + j * kThreads, n_ids - 1) / (uint32_t)p.k);
#pragma unroll
          for (int j = 0; j < kAhead; ++j)
            if (on[j] == 0) e[j] = kFull;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
          if (e[j] < (uint32_t)E) atomicAdd(&sc[e[j]], 1);
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
    const size_t slot = (size_t)blockIdx.x + s;
    float dot = 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sp[w * E + e];
      if constexpr (ONE) {
        p.counts[(size_t)s * E + e] = sc[e];
        p.prob_sum[(size_t)s * E + e] = v;
        dot = fmaf((float)sc[e], v, dot);
      } else {
        p.part[slot * E + e] = make_float2(v, __int_as_float(sc[e]));
      }
    }
    if constexpr (ONE) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
      __syncthreads();  // the probability sums are read
      if (lane == 0) sp[warp] = dot;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      float z = 0.0f;
      int c = 0;
      for (int w = 0; w < kWarps; ++w) {
        z += sz[w];
        c += sn[w];
      }
      if constexpr (ONE) {
        p.tokens[s] = c;
        if (c > 0) {
          float d = 0.0f;
          for (int w = 0; w < kWarps; ++w) d += sp[w];
          add(total, {d * ((float)E / ((float)p.k * (float)c)) / (float)c, z, c, 1});
        }
      } else {
        p.part_zn[slot] = make_float2(z, __int_as_float(c));
      }
    }
    __syncthreads();  // the shared sums are read before the next piece
    t0 = hi;
    ++s;
  }
  if constexpr (ONE) {
    for (; s < p.S; ++s) empty_sequence(p, s);
    if (threadIdx.x == 0) write_loss(p, total);
    return;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&p.err->ready, 1);
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

// Resident blocks of the backward on an SM: the grid is one wave of them (with a third of the blocks left for a
// second wave, 131072 tokens of 64 experts took 22 us).
constexpr int bwd_blocks(int V) { return V == 8 ? 2 : 3; }

// A warp owns a run of tokens; the f of the sequence at hand stays in
// registers and is read again where the sequence changes.
template <int G, int V, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, bwd_blocks(V)) balance_bwd_kernel(const BwdParams p) {
  constexpr int kTok = 32 / G;
  grid_wait();
  grid_launch_dependents();
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
      for (int v = 0; v < V; ++v) {
        const int c = 4 * (v * G + g);
        const int32_t* at = p.counts + (size_t)s * E + c;
        if (ALIGNED) {
          const int4 q = c < E ? __ldg(reinterpret_cast<const int4*>(at)) : make_int4(0, 0, 0, 0);
          f[4 * v] = fc * (float)q.x;
          f[4 * v + 1] = fc * (float)q.y;
          f[4 * v + 2] = fc * (float)q.z;
          f[4 * v + 3] = fc * (float)q.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[4 * v + i] = c + i < E ? fc * (float)__ldg(at + i) : 0.0f;
        }
      }
    }
    for (int t = t0 + sub; t - sub < hi; t += kTok) {
      float l[4 * V];
      const bool in = t < hi;
      load_row<G, V, ALIGNED>(p.logits + (size_t)(in ? t : t0) * E, g, E, in && inside, l);
      const float lse = in ? __ldg(p.lse + t) : 0.0f;
      const bool live = in && inside && (p.mask == nullptr || __ldg(p.mask + t) != 0);
      const bool some = lse != -INFINITY;  // a row of -inf alone has no probabilities
      // lse is rounded by 2^-24 of the logits' common offset, so exp(l - lse) is off by one factor in all of a row
      // (logits around 1000: 3e-5): their sum takes it out.
      float sum = 0.0f, dot = 0.0f;
#pragma unroll
      for (int i = 0; i < 4 * V; ++i) {
        l[i] = some && live ? exp_of(l[i] - lse) : 0.0f;
        sum += l[i];
        dot = fmaf(l[i], live ? f[i] : 0.0f, dot);
      }
      sum = group_sum<G>(sum);
      const float inv = some && live ? 1.0f / sum : 0.0f;
      dot = group_sum<G>(dot) * inv;
      const float zt = some ? zc * lse : 0.0f;
      if (!in) continue;
      float* row = p.d_logits + (size_t)t * E;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 4 * (v * G + g);
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = live ? l[4 * v + i] * inv * fmaf(bc, f[4 * v + i] - dot, zt) : 0.0f;
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
    t0 = hi;
  }
}

// Runs F<G, V, ALIGNED> for E columns.
template <template <int, int, bool> class F, typename... Args>
cudaError_t dispatch_columns(int E, Args... args) {
  const bool al = (E & 3) == 0;
#define E4B_BAL(G, V) return al ? F<G, V, true>::run(args...) : F<G, V, false>::run(args...)
  if (E <= 4) E4B_BAL(1, 1);
  if (E <= 8) E4B_BAL(1, 2);
  if (E <= 16) E4B_BAL(1, 4);
  if (E <= 32) E4B_BAL(2, 4);
  if (E <= 64) E4B_BAL(4, 4);
  if (E <= 128) E4B_BAL(8, 4);
  if (E <= 256) E4B_BAL(16, 4);
  if (E <= 512) E4B_BAL(32, 4);
  E4B_BAL(32, 8);
#undef E4B_BAL
}

template <int G, int V, bool ALIGNED>
struct RunFwd {
  static cudaError_t run(FwdParams p, int grid, cudaStream_t stream) {
    const int smem = (kWarps * p.E + p.E + 2 * kWarps) * 4;
    return launch_following(p.blocks == 1 ? balance_fwd_kernel<G, V, ALIGNED, true>
                                          : balance_fwd_kernel<G, V, ALIGNED, false>,
                            grid, kThreads, smem, 0, stream, p);
  }
};
template <int G, int V, bool ALIGNED>
struct RunBwd {
  static cudaError_t run(BwdParams p, int grid, cudaStream_t stream) {
    return launch_following(balance_bwd_kernel<G, V, ALIGNED>, grid, kThreads, 0, 0, stream, p);
  }
};

// Tokens that a warp's groups hold at a time.
int warp_tokens(int E) {
  int g = 1;
  while (g < 32 && 16 * g < E) g *= 2;
  return 32 / g;
}
// Token ranges: at least the tokens that a block's warps hold at a time, at most one wave of resident blocks.  (8192
// tokens of 128 experts, forward: 256 blocks of one round 10.3 us, 147 of two 12.4 us.)  Joining blocks: one an SM
// (30011 tokens of 256 experts in 37 sequences, forward: 64 20.6 us, 148 17.9 us).
constexpr int kJoinBlocks = 148;
constexpr int max_blocks(int E) { return 148 * fwd_blocks(E <= 512 ? 4 : 8); }
int balance_blocks(int T, int E) {
  const int at_once = kWarps * warp_tokens(E);
  const int b = (T + at_once - 1) / at_once;
  return b < max_blocks(E) ? b : max_blocks(E);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }
struct BalanceLayout {
  size_t part, part_zn, joined, total;
};
BalanceLayout balance_layout(int T, int E, int S) {
  const size_t slots = (size_t)balance_blocks(T, E) + S;
  BalanceLayout l;
  l.part = sizeof(DeviceError);
  l.part_zn = l.part + align256(slots * E * 8);
  l.joined = l.part_zn + align256(slots * 8);
  l.total = l.joined + align256(kJoinBlocks * sizeof(float4));
  return l;
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

cudaError_t launch_balance_fwd(const BalanceHost& h, void* ws, cudaStream_t stream) {
  const int want = balance_blocks(h.T, h.E);
  const BalanceLayout l = balance_layout(h.T, h.E, h.S);
  uint8_t* w = static_cast<uint8_t*>(ws);
  FwdParams p;
  p.per_block = (h.T + want - 1) / want;
  p.blocks = (h.T + p.per_block - 1) / p.per_block;
  p.logits = h.logits;
  p.ids = h.ids;
  p.offsets = h.offsets;
  p.mask = h.mask;
  p.err = reinterpret_cast<DeviceError*>(w);
  p.part = reinterpret_cast<float2*>(w + l.part);
  p.part_zn = reinterpret_cast<float2*>(w + l.part_zn);
  p.joined = reinterpret_cast<float4*>(w + l.joined);
  p.counts = h.counts;
  p.prob_sum = h.prob_sum;
  p.tokens = h.tokens;
  p.lse = h.lse;
  p.loss = h.loss;
  p.T = h.T;
  p.E = h.E;
  p.k = h.k;
  p.S = h.S;
  p.slices = (h.E + kSlice - 1) / kSlice;
  const int64_t items = (int64_t)h.S * p.slices;
  p.join_blocks = p.blocks == 1 ? 0 : (int)(items < kJoinBlocks ? items : kJoinBlocks);
  p.c_b = h.c_b;
  p.c_z = h.c_z;
  LaunchScope scope("balance_fwd", stream);
  return dispatch_columns<RunFwd>(h.E, p, p.blocks + p.join_blocks, stream);
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
  // runs of tokens: every resident warp takes one, at least the tokens it holds at a time
  const int64_t warps = (int64_t)num_sms * bwd_blocks(h.E > 512 ? 8 : 4) * kWarps;
  p.per_warp = (int)((h.T + warps - 1) / warps);
  const int at_once = warp_tokens(h.E);
  p.per_warp = (p.per_warp + at_once - 1) / at_once * at_once;
  const int64_t used = ((int64_t)h.T + p.per_warp - 1) / p.per_warp;
  const int grid = (int)((used + kWarps - 1) / kWarps);
  LaunchScope scope("balance_bwd", stream);
  return dispatch_columns<RunBwd>(h.E, p, grid, stream);
}

}  // namespace e4b
