// Small batches of the NF4 projection with adapters of many requests, mostly one
// launch each:
//
//   adapter_gemv_kernel:  y[t] = W x[t] + B[a] p[t], p[t] = s[a] A[a] x[t], for
//                         up to 16 tokens (8 of a large matrix);
//   adapter_split_kernel: the same for up to 256 tokens.
//
// What bounds them: reading the matrix (4.5 bits a weight) and each named
// adapter once, and latency: two dependent launches cost the host 9 us here and
// one 4.5 us, more than the GPU needs.  So the first blocks of the grid compute p
// while the others stream the matrix and wait for p (a counter in the workspace,
// bounded wait) only in their epilogue.  The blocks of p never wait and come
// first in the grid.
//
// For few tokens the products run on warp matrix instructions (m16n8k16): there is
// nothing for a 128-row UMMA tile to amortise its set-up over.  Above, reading x
// again for every 16 rows of W would cost more than W itself, and a UMMA takes 128
// rows of W (decoded into tensor memory) against all tokens at once, K split over a
// cluster whose partial sums meet through distributed shared memory.
//
// The sum over k may be taken in any order that both operands share, so in the
// warp products a lane takes 16 (W, x: 64) consecutive values of its row, and the
// elements it holds are declared to be the ones the instruction expects of it.
#include <math.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"
#include "launch.cuh"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokenTile = 8;
constexpr int kPlaces = 2 * 148;  // blocks of adapter_gemv_kernel at once

// Hand-over of p between the blocks of a launch.  signal_ready: the whole block, after its stores of p.
// wait_ready: one thread; false where the limit ran out.  leave: one thread, once the block has p.
__device__ __forceinline__ void signal_ready(DeviceError* err) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&err->ready, 1);
  }
}
__device__ __forceinline__ bool wait_ready(DeviceError* err, int blocks, long long timeout_ns, int site) {
  const long long c0 = clock64(), limit = wait_limit_cycles(timeout_ns);
  while (true) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(&err->ready) : "memory");
    if (v >= blocks) return true;
    if (clock64() - c0 > limit) {
      record_error(err, E4B_ERR_DEVICE_TIMEOUT, site);
      return false;
    }
  }
}
__device__ __forceinline__ void leave(DeviceError* err, int blocks) {
  if (atomicAdd(&err->left, 1) == blocks - 1) {
    err->ready = 0;
    err->left = 0;
  }
}

// D (16 x 8) += A (16 x 16) B (16 x 8), bf16 inputs, float32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes, or zeros where `ok` is false (nothing is read then).  Volatile, so that a batch of loads written
// ahead of the instructions that use them is issued ahead of them: left to the compiler, they were paired with
// their uses and few were in flight.
__device__ __forceinline__ uint4 ldg16(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "setp.ne.b32 q, %5, 0;\n"
      "mov.u32 %0, 0;\n"
      "mov.u32 %1, 0;\n"
      "mov.u32 %2, 0;\n"
      "mov.u32 %3, 0;\n"
      "@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n"
      "}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p), "r"((int)ok));
  return v;
}

// ----------------------------------------------------------------------------
// 16 ranks of an adapter against up to eight tokens, over [k_lo, k_hi)
// ----------------------------------------------------------------------------
// The block's warps split the range, lanes read A and x straight from global
// memory; every warp leaves its partial sums in red[warp][rank][token].  t: the
// token of this lane's column (-1: none); k_lo a multiple of 32.
template <int WARPS>
__device__ __forceinline__ void low_rank_tile(const uint16_t* x, const uint16_t* A, int K, int r, int a, int t, int j0,
                                              int k_lo, int k_hi, float (*red)[16][kTokenTile + 1]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const bool tok = t >= 0, lo = j0 + g < r, hi = j0 + g + 8 < r;
  const uint16_t* xr = x + (tok ? (size_t)t * K : 0) + 8 * q;
  const uint16_t* a0 = A + ((size_t)a * r + (lo ? j0 + g : 0)) * K + 8 * q;
  const uint16_t* a1 = A + ((size_t)a * r + (hi ? j0 + g + 8 : 0)) * K + 8 * q;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  // 32 values of k a step: lane q of a row holds 8 of them, two instructions' worth.  Four steps' loads go out
  // together.
  constexpr int kAhead = 4;
  for (int k0 = k_lo + warp * 32; k0 < k_hi; k0 += WARPS * 32 * kAhead) {
    uint4 w0[kAhead], w1[kAhead], xv[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * WARPS * 32;
      w0[i] = ldg16(a0 + k, lo && k < k_hi);
      w1[i] = ldg16(a1 + k, hi && k < k_hi);
      xv[i] = ldg16(xr + k, tok && k < k_hi);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      mma_bf16(acc, w0[i].x, w1[i].x, w0[i].y, w1[i].y, xv[i].x, xv[i].y);
      mma_bf16(acc, w0[i].z, w1[i].z, w0[i].w, w1[i].w, xv[i].z, xv[i].w);
    }
  }
  red[warp][g][2 * q] = acc[0];
  red[warp][g][2 * q + 1] = acc[1];
  red[warp][g + 8][2 * q] = acc[2];
  red[warp][g + 8][2 * q + 1] = acc[3];
}

// ----------------------------------------------------------------------------
// y for up to 16 tokens: 16 rows of W at a time, K split over the block's warps
// ----------------------------------------------------------------------------
// Blocks stay for several units of rows, the next unit's codes in flight while one
// ends and p read once: 4096 -> 14336, 1 token 20.2 us, 8 tokens 24.6 us (a block a
// unit: 9 and 13% more).  1 token at 2048 -> 4096 takes 8.1 us alone and 5.9 us after
// another, the chain of loads and waits; on the large matrix the byte permutes of the
// decoding keep the ALU pipe busy for 58% of the active cycles, 11 us, and what is left
// is between the steps.  Decoding by a table of byte pairs in shared memory instead
// takes 10% less at 1 token, but 23% more at 8, whose rows of x come through the same
// pipe (L1 77% busy there as it is).
// The blocks of p take (token, 16 ranks, share of K) each; with few of them K is
// split (kq shares, added in order by the readers), since one block's loads
// would be the longest chain of the launch.
struct GemvParams {
  const int32_t* ids;
  const uint16_t* x;
  const uint8_t* nf4;
  const float* absmax;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  float* part;  // [kq, T, r] shares of A x
  uint16_t* y;
  DeviceError* err;
  long long timeout_ns;
  int T, K, N, n, r;
  int kq, p_blocks;
};

template <int NT>  // tiles of 8 tokens
__global__ void __launch_bounds__(kThreads, 2) adapter_gemv_kernel(const GemvParams p) {
  __shared__ float red[2][kWarps * 8 * NT * 17];  // a unit's partial sums, in turn; a block of p: [warp][16][9]
  static_assert(2 * 8 * NT * 17 >= 16 * 9, "a block of p fits");
  grid_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  if ((int)blockIdx.x < p.p_blocks) {
    const int slices = (p.r + 15) / 16;
    const int share = (int)blockIdx.x % p.kq, item = (int)blockIdx.x / p.kq;
    const int t = item / slices, j0 = (item - t * slices) * 16;
    const int a = __ldg(p.ids + t);
    if ((uint32_t)a < (uint32_t)p.n) {
      float(*tile)[16][kTokenTile + 1] = reinterpret_cast<float(*)[16][kTokenTile + 1]>(red[0]);
      const int blocks32 = p.K / 32;
      low_rank_tile<kWarps>(p.x, p.A, p.K, p.r, a, g == 0 ? t : -1, j0, share * blocks32 / p.kq * 32,
                            (share + 1) * blocks32 / p.kq * 32, tile);
      __syncthreads();
      if (tid < 16 && j0 + tid < p.r) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += tile[w][tid][0];
        p.part[((size_t)share * p.T + t) * p.r + j0 + tid] = v;
      }
    }
    signal_ready(p.err);
    return;
  }
  // A unit is 16 rows of W; a step of a warp is 256 values of k, one NF4 block of 64 a lane and row.
  const int units = (p.N + 15) / 16, step = (int)gridDim.x - p.p_blocks;
  const uint16_t* xr[NT];
  bool tok[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    tok[i] = 8 * i + g < p.T;
    xr[i] = p.x + (tok[i] ? (size_t)(8 * i + g) * p.K : 0) + 64 * q;
  }
  const Nf4Shift ks = nf4_shift_consts();
  struct Raw {
    uint4 a[2], b[2];
    float ma, mb;
  };
  auto load = [&](int unit, int k0) -> Raw {
    Raw w;
    const bool in = k0 + 64 * q < p.K;  // K is a multiple of 64: the last step may be short of blocks
    const int ra = 16 * unit + g, rb = ra + 8;
    const bool lo = in && ra < p.N, hi = in && rb < p.N;
    const size_t at = (size_t)(k0 / 2 + 32 * q), sat = (size_t)(k0 / 64 + q);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w.a[h] = ldg16(p.nf4 + (lo ? (size_t)ra * (p.K / 2) + at + 16 * h : 0), lo);
      w.b[h] = ldg16(p.nf4 + (hi ? (size_t)rb * (p.K / 2) + at + 16 * h : 0), hi);
    }
    w.ma = lo ? __ldg(p.absmax + (size_t)ra * (p.K / 64) + sat) : 0.0f;
    w.mb = hi ? __ldg(p.absmax + (size_t)rb * (p.K / 64) + sat) : 0.0f;
    return w;
  };
  const int t = tid >> 4, row = tid & 15;  // this thread's output of a unit
  uint32_t a = 0xffffffffu;
  if (t < p.T) a = (uint32_t)__ldg(p.ids + t);
  const bool adapted = a < (uint32_t)p.n;
  __shared__ float ps[8 * NT][E4B_MAX_RANK + 4];
  __shared__ int have;
  bool first = true;
  int buf = 0;
  int unit = (int)blockIdx.x - p.p_blocks;
  Raw next = load(unit, warp * 256);
  for (; unit < units; unit += step, buf ^= 1) {
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    for (int k0 = warp * 256; k0 < p.K; k0 += kWarps * 256) {
      const Raw w = next;
      const bool in = k0 + 64 * q < p.K;
      // x of both halves of the block at once, or (two tiles: the registers) one after the other
      constexpr int kXHalves = NT == 1 ? 2 : 1;
      uint4 xv[NT][4 * kXHalves];
      auto load_x = [&](int h) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            xv[j][4 * (h % kXHalves) + c] = ldg16(xr[j] + k0 + 32 * h + 8 * c, in && tok[j]);
      };
      load_x(0);
      if (kXHalves == 2) load_x(1);
      // the next step's codes, or the next unit's first (rows past N read as zeros)
      const bool more = k0 + kWarps * 256 < p.K;
      next = load(more ? unit : unit + step, more ? k0 + kWarps * 256 : warp * 256);
      const Nf4Planes pa = nf4_block_planes(w.ma), pb = nf4_block_planes(w.mb);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t ca[4] = {w.a[h].x, w.a[h].y, w.a[h].z, w.a[h].w};
        const uint32_t cb[4] = {w.b[h].x, w.b[h].y, w.b[h].z, w.b[h].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t da[4], db[4];
          nf4_decode_word(ca[c], pa, ks, da);
          nf4_decode_word(cb[c], pb, ks, db);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 v = xv[j][4 * (h % kXHalves) + c];
            mma_bf16(acc[j], da[0], db[0], da[1], db[1], v.x, v.y);
            mma_bf16(acc[j], da[2], db[2], da[3], db[3], v.z, v.w);
          }
        }
        if (h == 0 && kXHalves == 1) load_x(1);
      }
    }
    float(*sums)[8 * NT][17] = reinterpret_cast<float(*)[8 * NT][17]>(red[buf]);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      sums[warp][8 * i + 2 * q][g] = acc[i][0];
      sums[warp][8 * i + 2 * q + 1][g] = acc[i][1];
      sums[warp][8 * i + 2 * q][g + 8] = acc[i][2];
      sums[warp][8 * i + 2 * q + 1][g + 8] = acc[i][3];
    }
    // One output a thread: its adapter's row of B is fetched before p is waited for.
    const int n = 16 * unit + row;
    const bool mine = t < p.T && n < p.N;
    uint4 bw[E4B_MAX_RANK / 8];
#pragma unroll
    for (int j = 0; j < E4B_MAX_RANK / 8; ++j)
      bw[j] = ldg16(p.B + ((size_t)(adapted ? a : 0) * p.N + (mine ? n : 0)) * p.r + (8 * j < p.r ? 8 * j : 0),
                    adapted && mine && 8 * j < p.r);
    if (first && tid == 0) have = wait_ready(p.err, p.p_blocks, p.timeout_ns, 640);
    __syncthreads();
    if (first) {
      if (!have) return;
      first = false;
      if (tid == 0) leave(p.err, step);
      // p[t, j] = s[a] sum of the shares, 16 threads a token
      if (adapted) {
        const float sc = __ldg(p.scale + a);
        for (int j = 4 * row; j < p.r; j += 64) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int s = 0; s < p.kq; ++s) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(p.part + ((size_t)s * p.T + t) * p.r + j));
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
          }
          *reinterpret_cast<float4*>(&ps[t][j]) = make_float4(sc * v.x, sc * v.y, sc * v.z, sc * v.w);
        }
      }
      __syncwarp();  // a token's 16 threads are of one warp
    }
    if (mine) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sums[w][t][row];
      if (adapted) {
#pragma unroll
        for (int j = 0; j < E4B_MAX_RANK / 8; ++j) {
          if (8 * j >= p.r) break;
          const uint32_t b4[4] = {bw[j].x, bw[j].y, bw[j].z, bw[j].w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v = fmaf(bf16lo_to_f32(b4[c]), ps[t][8 * j + 2 * c], v);
            v = fmaf(bf16hi_to_f32(b4[c]), ps[t][8 * j + 2 * c + 1], v);
          }
        }
      }
      const __nv_bfloat16 h = __float2bfloat16_rn(v);
      p.y[(size_t)t * p.N + n] = *reinterpret_cast<const uint16_t*>(&h);
    }
  }
}

// ----------------------------------------------------------------------------
// y for up to 256 tokens: 128 rows of W x all tokens x a share of K per block
// ----------------------------------------------------------------------------
// After the blocks of p (or under a launch of p of its own): warp 0 loads x tiles
// (TMA), warp 1 owns tensor memory and issues the UMMAs, warp 2 sorts the tokens
// into tiles of eight of one adapter, warps 4-15 are three decode teams that take
// the k-chunks round robin: a thread owns a row of W, reads 32 bytes of codes and a
// scale a chunk straight into registers two of its chunks ahead, and writes the
// decoded row to the A buffer in tensor memory.  Each of the cluster's S blocks then
// owns 128 / S of the rows: the partial sums are stored into their owners' shared
// memory (over the x tiles; reading them from there instead took 4.7 us at 256
// tokens, one round trip after another), added, and the adapters' part is added in
// the fragment layout of the warp instruction, tile by tile, so that no adapter's
// values meet another's tokens.  256 tokens, 4096 -> 4096, 32 adapters of rank 32:
// 22.3 us with inputs that stay in L2, 25.6 us with others in every call, bound by the
// L2 reads of x (64 KB/us a block; all of x for every 128 rows of W, 64 MB) and the
// exchange of shares; 57 tokens, 2048 -> 512: 12 us, the chain p, hand-over, join; 64
// tokens, 4096 -> 14336, 16 adapters: 30 us, the ALU pipe (the decode's byte permutes)
// 95% busy in the loop.  A fourth team, or coalesced
// code loads, change nothing there; a quarter of the words by a table of byte pairs
// gains 4%.
namespace ads {
constexpr int BM = 128, BK = 64;
constexpr int kXStages = 4, kTeams = 3, kABufs = 2 * kTeams, kACols = BK / 2;
constexpr int kThreadsSplit = 512;
constexpr int kAOff = 256;             // TMEM columns: accumulator [0, 256), A buffers behind
constexpr int kTmemCols = 512;
constexpr int kBarBytes = 256;
constexpr int kListBytes = (9 * kAdapterSmallTokens + E4B_MAX_ADAPTERS) * 2;
inline int ring_bytes(int nt, int S) {  // x tiles, then the S shares of 128 / S rows (4 floats of padding a token)
  const int x = kXStages * nt * BK * 2, part = nt * (BM + 4 * S) * 4;
  return ((x > part ? x : part) + 1023) / 1024 * 1024;
}
constexpr int kMaxSmem = 232448;
static_assert(kAOff + kABufs * kACols <= kTmemCols, "TMEM budget");
}  // namespace ads

struct SplitParams {
  const uint8_t* nf4;
  const float* absmax;
  const uint16_t* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  uint16_t* p;         // [T, 2, r] pairs
  const int32_t* ids;
  uint16_t* y;
  DeviceError* err;
  long long timeout_ns;
  int T, NT, K, N, n, r;  // NT: T rounded up to 16
  int ring;               // bytes of the x ring / partial sums
  int p_blocks;           // blocks of p, ahead of the others (whole clusters); 0: p has a launch of its own
};

// Shared memory of a block of p of kWarps warps.
constexpr int kLowRankBytes = kWarps * 16 * (kTokenTile + 1) * 4 + (3 * kAdapterSmallTokens + kTokenTile + kWarps) * 2;

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// As ldg16, from L2: the launch that wrote it may have run beside this one.
__device__ __forceinline__ uint4 ldcg16(const void* p, bool ok) {
  uint4 v;
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "setp.ne.b32 q, %5, 0;\n"
      "mov.u32 %0, 0;\n"
      "mov.u32 %1, 0;\n"
      "mov.u32 %2, 0;\n"
      "mov.u32 %3, 0;\n"
      "@q ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n"
      "}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "l"(p), "r"((int)ok)
      : "memory");
  return v;
}

// p for the split kernel: the tokens of an adapter in tiles of up to eight, in token order; an item is (tile, 16
// ranks), and the `blocks` blocks of kW warps take the items in turn.
template <int kW>
__device__ __forceinline__ void split_low_rank(uint8_t* smem, const SplitParams& p, int blocks) {
  static_assert(kAdapterSmallTokens <= 32 * kW, "a token a thread");
  float(*red)[16][kTokenTile + 1] = reinterpret_cast<float(*)[16][kTokenTile + 1]>(smem);
  int16_t* ids = reinterpret_cast<int16_t*>(red + kW);    // [kAdapterSmallTokens] -1: no adapter
  int16_t* first = ids + kAdapterSmallTokens;             // first tokens of the tiles
  int16_t* ranks = first + kAdapterSmallTokens;           // and their ranks
  int16_t* tok = ranks + kAdapterSmallTokens;             // [8] tokens of the item's tile
  int16_t* warp_tiles = tok + kTokenTile;                 // [kW]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2;
  int a = -1;
  if (tid < kAdapterSmallTokens) {
    const uint32_t id = tid < p.T ? (uint32_t)__ldg(p.ids + tid) : kFull;
    a = id < (uint32_t)p.n ? (int)id : -1;
    ids[tid] = (int16_t)a;
  }
  __syncthreads();
  // this token's rank among its adapter's: a warp counts eight earlier tokens a read
  int rank = 0;
  if (a >= 0) {
    const uint32_t want = (uint32_t)a * 0x10001u;
    for (int i = 0; i < tid / 8; ++i) {
      const uint4 w = reinterpret_cast<const uint4*>(ids)[i];
      rank += __popc(__vcmpeq2(w.x, want) & 0x10001u) + __popc(__vcmpeq2(w.y, want) & 0x10001u) +
              __popc(__vcmpeq2(w.z, want) & 0x10001u) + __popc(__vcmpeq2(w.w, want) & 0x10001u);
    }
    for (int i = tid / 8 * 8; i < tid; ++i) rank += ids[i] == a;
  }
  const bool opens = a >= 0 && rank % kTokenTile == 0;
  const uint32_t b = __ballot_sync(kFull, opens);
  if (lane == 0) warp_tiles[warp] = (int16_t)__popc(b);
  __syncthreads();
  int at = __popc(b & ((1u << lane) - 1)), n_tiles = 0;
  for (int w = 0; w < kW; ++w) {
    if (w < warp) at += warp_tiles[w];
    n_tiles += warp_tiles[w];
  }
  if (opens) {
    first[at] = (int16_t)tid;
    ranks[at] = (int16_t)rank;
  }
  const int slices = (p.r + 15) / 16;
  for (int item = (int)blockIdx.x; item < n_tiles * slices; item += blocks) {
    const int tile = item / slices, j0 = (item - tile * slices) * 16;
    __syncthreads();  // the list; the last item's tokens and sums are read
    if (tid < kTokenTile) tok[tid] = -1;
    const int ad = ids[first[tile]];
    __syncthreads();
    const int d = rank - ranks[tile];  // the tile's first token and the next seven of its adapter
    if (a == ad && d >= 0 && d < kTokenTile) tok[d] = (int16_t)tid;
    __syncthreads();
    low_rank_tile<kW>(p.x, p.A, p.K, p.r, ad, tok[g], j0, 0, p.K, red);
    __syncthreads();
    if (tid < 16 * kTokenTile) {
      const int j = tid & 15, c = tid >> 4, t = tok[c];
      if (t >= 0 && j0 + j < p.r) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kW; ++w) v += red[w][j][c];
        uint32_t high, low;
        split_bf16x2(__ldg(p.scale + ad) * v, 0.0f, high, low);
        uint16_t* at = p.p + (size_t)t * 2 * p.r + j0 + j;
        at[0] = (uint16_t)high;
        at[p.r] = (uint16_t)low;
      }
    }
  }
}

// The same as a launch of its own, which the products start under: with 64 registers and 256 threads a block fits
// beside one of theirs.
__global__ void __launch_bounds__(kThreads, 4) adapter_low_rank_kernel(const SplitParams p) {
  __shared__ __align__(16) uint8_t smem[kLowRankBytes];
  grid_wait();
  grid_launch_dependents();
  split_low_rank<kWarps>(smem, p, (int)gridDim.x);
}

template <int S, bool WIDE>  // blocks of a cluster, the shares of K; r > 32
__global__ void __launch_bounds__(ads::kThreadsSplit + 128, 1)  // 96 registers: the launch of p beside
    adapter_split_kernel(const __grid_constant__ CUtensorMap map_x, const SplitParams p) {
  using namespace ads;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  if ((int)blockIdx.x < p.p_blocks) {
    grid_wait();
    grid_launch_dependents();
    split_low_rank<kThreadsSplit / 32>(smem, p, p.p_blocks);
    signal_ready(p.err);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ring);
  uint64_t* x_full = bars;                  // [kXStages]
  uint64_t* x_empty = x_full + kXStages;    // [kXStages]
  uint64_t* a_ready = x_empty + kXStages;   // [kABufs] a team's decoded chunk is in tensor memory (4 warps)
  uint64_t* a_empty = a_ready + kABufs;     // [kABufs]
  uint64_t* accfull = a_empty + kABufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accfull + 1);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(accfull + 2);
  int32_t* n_tiles = reinterpret_cast<int32_t*>(accfull + 3);
  int16_t* tile_ad = reinterpret_cast<int16_t*>(smem + p.ring + kBarBytes);  // [kAdapterSmallTokens]
  int16_t* tile_tok = tile_ad + kAdapterSmallTokens;                         // eight a tile, -1: none
  int16_t* count = tile_tok + kTokenTile * kAdapterSmallTokens;              // [n]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)(blockIdx.x % S), n0 = (int)((blockIdx.x - p.p_blocks) / S) * BM;
  const int chunks = p.K / BK;
  const int k_lo = rank * chunks / S, nc = (rank + 1) * chunks / S - k_lo;
  if (tid == 0) {
    for (int s = 0; s < kXStages; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&x_empty[s], 1);
    }
    for (int b = 0; b < kABufs; ++b) {
      mbar_init(&a_ready[b], 4);
      mbar_init(&a_empty[b], 1);
    }
    mbar_init(accfull, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (p.p_blocks > 0) {  // else the launch of p has waited, and only p is still to come
    grid_wait();
    grid_launch_dependents();
  }
  const int x_bytes = p.NT * BK * 2;
  bool done = false;  // (teams) the accumulator is complete

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&map_x);
      uint32_t issued = 0, last_par = 0;
      bool ok = true;
      for (int i = 0; i < nc; ++i) {
        const uint32_t s = i % kXStages, ph = (i / kXStages) & 1;
        if (!(ok = mbar_wait(&x_empty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 610))) break;
        mbar_arrive_expect_tx(&x_full[s], (uint32_t)x_bytes);
        tma_load_2d(smem + s * x_bytes, &map_x, &x_full[s], (k_lo + i) * BK, 0);
        issued |= 1u << s;
        last_par = (last_par & ~(1u << s)) | (ph << s);
      }
      if (!ok)
        for (int s = 0; s < kXStages; ++s)
          if (issued & (1u << s)) {
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&x_full[s], (last_par >> s) & 1u) &&
                   (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
            }
          }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one_sync()) {
      const uint32_t idesc = make_idesc_bf16(BM, p.NT, false, false);
      const uint64_t xdesc0 = make_sdesc(smem_u32(smem), 16, 1024, kSw128);
      for (int i = 0; i < nc; ++i) {
        const uint32_t b = i % kABufs, s = i % kXStages;
        if (!mbar_wait(&a_ready[b], (i / kABufs) & 1, ctl, p.err, p.timeout_ns, 620)) break;
        if (!mbar_wait(&x_full[s], (i / kXStages) & 1, ctl, p.err, p.timeout_ns, 621)) break;
        tc_fence_after();
        const uint64_t xd = xdesc0 + (uint64_t)((s * x_bytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          umma_bf16_ta(tmem, tmem + kAOff + b * kACols + 8 * kk, xd + 2 * kk, idesc, (i > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&a_empty[b]);
        umma_commit(&x_empty[s]);
      }
      // also where a wait ran out: nothing issued is left running when this wait ends
      umma_commit(accfull);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(accfull, 0) && (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- token tiles: a stable counting sort of the tokens by adapter, in the shadow of the products
    for (int i = lane; i < p.n; i += 32) count[i] = 0;
    __syncwarp();
    constexpr int kRounds = kAdapterSmallTokens / 32;
    int16_t ad[kRounds], pos[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int t = 32 * i + lane;
      const uint32_t a = t < p.T ? (uint32_t)__ldg(p.ids + t) : kFull;
      ad[i] = a < (uint32_t)p.n ? (int16_t)a : (int16_t)-1;
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const uint32_t same = __match_any_sync(kFull, (int)ad[i]);
      const int rank_in = __popc(same & ((1u << lane) - 1));
      pos[i] = ad[i] >= 0 ? (int16_t)(count[ad[i]] + rank_in) : (int16_t)0;
      __syncwarp();
      if (ad[i] >= 0 && rank_in == 0) count[ad[i]] += (int16_t)__popc(same);
      __syncwarp();
    }
    // an adapter's first tile; lane l owns adapters l m ..
    const int m = (p.n + 31) / 32;
    int sum = 0;
    for (int i = lane * m; i < min(p.n, lane * m + m); ++i) sum += (count[i] + kTokenTile - 1) / kTokenTile;
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    const int total = __shfl_sync(kFull, incl, 31);
    for (int i = lane; i < total * kTokenTile; i += 32) tile_tok[i] = -1;
    int base = incl - sum;
    for (int i = lane * m; i < min(p.n, lane * m + m); ++i) {
      const int tiles = (count[i] + kTokenTile - 1) / kTokenTile;
      count[i] = (int16_t)base;
      for (int j = 0; j < tiles; ++j) tile_ad[base++] = (int16_t)i;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (ad[i] >= 0) tile_tok[count[ad[i]] * kTokenTile + pos[i]] = (int16_t)(32 * i + lane);
    if (lane == 0) *n_tiles = total;
  } else if (warp >= 4) {
    const int team = (warp - 4) >> 2, row = n0 + 32 * (warp & 3) + lane;
    const bool valid = row < p.N;
    const uint4* codes = reinterpret_cast<const uint4*>(p.nf4 + (size_t)(valid ? row : 0) * (p.K / 2));
    const float* scales = p.absmax + (size_t)(valid ? row : 0) * chunks;
    const Nf4Shift ks = nf4_shift_consts();
    const uint32_t a_base = tmem + kAOff + ((uint32_t)(32 * (warp & 3)) << 16);
    struct Raw {
      uint4 a, b;
      float m;
    };
    auto load = [&](int i) -> Raw {
      Raw w;
      const bool go = valid && i < nc;  // rows past the matrix: a zero scale, zero weights
      w.a = ldg16(codes + 2 * (k_lo + i), go);
      w.b = ldg16(codes + 2 * (k_lo + i) + 1, go);
      w.m = go ? __ldg(scales + k_lo + i) : 0.0f;
      return w;
    };
    Raw w0 = load(team), w1 = load(team + kTeams);
    for (int i = team; i < nc; i += kTeams) {
      const Raw w2 = load(i + 2 * kTeams);
      const uint32_t b = i % kABufs;
      const uint32_t cw[8] = {w0.a.x, w0.a.y, w0.a.z, w0.a.w, w0.b.x, w0.b.y, w0.b.z, w0.b.w};
      const Nf4Planes pl = nf4_block_planes(w0.m);
      uint32_t v[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) nf4_decode_word(cw[c], pl, ks, &v[4 * c]);
      if (!__all_sync(kFull, mbar_wait(&a_empty[b], ((i / kABufs) & 1) ^ 1, ctl, p.err, p.timeout_ns, 630))) break;
      tc_fence_after();
      tmem_st32(a_base + b * kACols, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_ready[b]);
      w0 = w1;
      w1 = w2;
    }
    done = __all_sync(kFull, mbar_wait(accfull, 0, ctl, p.err, p.timeout_ns, 631));
  }
  __syncwarp();
  cluster_sync();  // no block's UMMAs read its x tiles any more
  // Partial sums into the shared memory of the block that owns the row, [share][token][row]: a lane holds a row
  // of the accumulator, so a store writes whole runs of rows.  Team by team 16 columns.
  constexpr int kRows = BM / S, kPitch = kRows + 4;
  const int rank0 = rank * kRows;
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= 4 && done) {
    tc_fence_after();
    const int team = (warp - 4) >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t to = mapa_shared(smem_u32(part + (size_t)rank * p.NT * kPitch + row % kRows), (uint32_t)(row / kRows));
    for (int c = 16 * team; c < p.NT; c += 16 * kTeams) {
      float v[16];
      tmem_ld16(tmem + c + ((uint32_t)(32 * (warp & 3)) << 16), v);
#pragma unroll
      for (int i = 0; i < 16; ++i) st_cluster_f32(to + (uint32_t)((c + i) * kPitch * 4), v[i]);
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();  // every share is in place
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // The shares of K are added in order.
  if constexpr (S > 1) {
    for (int i = tid; i < p.T * (kRows / 4); i += kThreadsSplit) {
      float4* at = reinterpret_cast<float4*>(part + (i / (kRows / 4)) * kPitch + 4 * (i % (kRows / 4)));
      float4 v = at[0];
#pragma unroll
      for (int s = 1; s < S; ++s) {
        const float4 w = at[(size_t)s * p.NT * (kPitch / 4)];
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      at[0] = v;
    }
  }
  if (p.p_blocks == 0) {
    grid_wait();  // p, from the launch ahead
    grid_launch_dependents();
    __syncthreads();
  } else {
    if (tid == 0) ctl->pad = wait_ready(p.err, p.p_blocks, p.timeout_ns, 641);
    __syncthreads();
    if (!ctl->pad) return;
    if (tid == 0) leave(p.err, (int)gridDim.x - p.p_blocks);
  }
  // The adapters' part: item = (tile of 8 tokens of one adapter, group of 16 rows), several items' fragments of B and p
  // fetched together.
  {
    constexpr int kGroupsOf16 = kRows / 16, kItemWarps = kThreadsSplit / 32, kC = WIDE ? 2 : 1;
    const int g = lane >> 2, q = lane & 3;
    const int items = *n_tiles * kGroupsOf16;
    struct Low {
      uint4 b0[kC], b1[kC], p[kC], p_low[kC];
    };
    auto fetch = [&](int item) -> Low {
      Low w;
      const int tile = item / kGroupsOf16, row = n0 + rank0 + 16 * (item % kGroupsOf16);
      const bool on = item < items && row < p.N;
      const int a = on ? tile_ad[tile] : 0, t = on ? tile_tok[tile * kTokenTile + g] : -1;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int j = 32 * c + 8 * q;
        const bool go = on && j < p.r;
        const uint16_t* b = p.B + ((size_t)a * p.N + (go ? row + g : 0)) * p.r + (go ? j : 0);
        w.b0[c] = ldg16(b, go);
        w.b1[c] = ldg16(b + 8 * p.r, go && row + 8 < p.N);  // N is a multiple of 8
        const uint16_t* pt = p.p + (size_t)(t >= 0 ? t : 0) * 2 * p.r + (go ? j : 0);
        w.p[c] = ldcg16(pt, go && t >= 0);
        w.p_low[c] = ldcg16(pt + p.r, go && t >= 0);
      }
      return w;
    };
    constexpr int kAtOnce = WIDE ? 2 : 4;
    for (int first = warp; first < items; first += kAtOnce * kItemWarps) {
      Low w[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) w[i] = fetch(first + i * kItemWarps);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int item = first + i * kItemWarps;
        if (item >= items) break;
        const int tile = item / kGroupsOf16, lrow = 16 * (item % kGroupsOf16);
        const int t0 = tile_tok[tile * kTokenTile + 2 * q], t1 = tile_tok[tile * kTokenTile + 2 * q + 1];
        float* c0 = part + (t0 < 0 ? 0 : t0) * kPitch + lrow + g;
        float* c1 = part + (t1 < 0 ? 0 : t1) * kPitch + lrow + g;
        float d[4] = {c0[0], c1[0], c0[8], c1[8]};
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          mma_bf16(d, w[i].b0[c].x, w[i].b1[c].x, w[i].b0[c].y, w[i].b1[c].y, w[i].p[c].x, w[i].p[c].y);
          mma_bf16(d, w[i].b0[c].z, w[i].b1[c].z, w[i].b0[c].w, w[i].b1[c].w, w[i].p[c].z, w[i].p[c].w);
          mma_bf16(d, w[i].b0[c].x, w[i].b1[c].x, w[i].b0[c].y, w[i].b1[c].y, w[i].p_low[c].x, w[i].p_low[c].y);
          mma_bf16(d, w[i].b0[c].z, w[i].b1[c].z, w[i].b0[c].w, w[i].b1[c].w, w[i].p_low[c].z, w[i].p_low[c].w);
        }
        if (t0 >= 0) c0[0] = d[0], c0[8] = d[2];
        if (t1 >= 0) c1[0] = d[1], c1[8] = d[3];
      }
    }
  }
  __syncthreads();
  // y, eight rows (16 bytes) of a token a thread; N is a multiple of 8
  for (int i = tid; i < p.T * (kRows / 8); i += kThreadsSplit) {
    const int t = i / (kRows / 8), lrow = 8 * (i % (kRows / 8));
    const float4 u = *reinterpret_cast<const float4*>(part + t * kPitch + lrow);
    const float4 v = *reinterpret_cast<const float4*>(part + t * kPitch + lrow + 4);
    if (n0 + rank0 + lrow < p.N)
      *reinterpret_cast<uint4*>(p.y + (size_t)t * p.N + n0 + rank0 + lrow) =
          make_uint4(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w), pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  }
}

}  // namespace

// Warp products for up to eight tokens, and for up to 16 of a matrix below 2^24 weights: with two token tiles their
// reads of x and their decoding for every 16 rows cost more than the UMMA kernel's set-up (16 tokens, warp products
// and UMMAs: 2048 -> 4096 9.2 and 10.6 us, 4096 -> 4096 14.4 and 15.2 us, 4096 -> 14336 42.6 and 29.7 us; 8 tokens
// at 4096 -> 14336 24.6 and 26.9 us).
bool adapter_gemv_serves(int T, int K, int N) {
  return T <= kTokenTile || (T <= 2 * kTokenTile && (int64_t)K * N < (1 << 24));
}

// Shares of K of the blocks of p of the warp products: as many as leave every block of the launch a place (two an
// SM; with 24 of 320 blocks in a second wave, 16 tokens at 2048 -> 4096 take 10.5 us, not 9.2).
int adapter_gemv_shares(int T, int r, int N) {
  const int items = T * ((r + 15) / 16), places = kPlaces - (N + 15) / 16;
  return 4 * items <= places ? 4 : (2 * items <= places ? 2 : 1);
}

// The shares S of K and the blocks of p, by an estimate in microseconds of what bounds each part: a block of p reads
// A at 90 KB/us and needs 1.7 us an item (2.5 us with 8 warps); a chunk of the product costs 0.3 us of decoding or its
// x tile at 80 KB/us; shares travel at 27 KB/us a block; one SM holds one block, and clusters of 2, 4, 8 find 74, 33,
// 15 places.  Either p has places of its own beside the products, or a launch of its own ahead of them (2 us).  Only
// the GPU's time counts: with the host's for two launches held against the second one, 20 of 189 sizes measured took
// up to a quarter longer, replayed from a graph and called alike (p in the launch and in its own, replayed: 57 tokens
// of 32 adapters of rank 32 at 4096 -> 4096 17.9 and 15.4 us, 17 tokens at 2048 -> 4096 11.2 and 9.9 us, 57 of 64 of
// rank 64 at 2048 -> 512 11.1 and 11.7 us).  S measured: 128 tokens at 2048 -> 2048, S = 8 (16 clusters in 15 places)
// 26.7 us, S = 4 14.4 us.
struct SplitPlan {
  int S, p_blocks;
  bool own;  // p in a launch of its own
};
static SplitPlan split_plan(const AdapterProjHost& h, int NT, int tiles, int chunks) {
  const int slices = (h.r + 15) / 16, named = h.T < h.n ? h.T : h.n;
  const int items = (h.T / kTokenTile + named < h.T ? h.T / kTokenTile + named : h.T) * slices;
  const float a_kb = (float)named * h.r * h.K * 2e-3f;
  auto p_time = [&](int blocks, float turn) {
    const float read = a_kb / (90.0f * blocks), turns = turn * ((items + blocks - 1) / blocks);
    return 1.5f + (read > turns ? read : turns);
  };
  SplitPlan best{1, 1, true};
  float best_time = 1e30f;
  const int places[4] = {148, 74, 33, 15};
  for (int i = 0; i < 4 && (i == 0 || chunks >= (2 << i)); ++i) {
    const int S = 1 << i;
    const float x_time = NT * 0.128f / 80.0f, step = x_time > 0.3f ? x_time : 0.3f;
    const float product = 2.5f + step * ((chunks + S - 1) / S) + NT * 0.512f * (S - 1) / S / 27.0f;
    const int turns = (tiles + places[i] - 1) / places[i];
    for (int own = 0; own < 2; ++own) {
      int blocks = own ? 148 : (places[i] - tiles) * S;
      const int most = own ? items : (items + S - 1) / S * S;
      if (blocks > most) blocks = most;
      if (blocks <= 0) continue;
      const float pt = p_time(blocks, own ? 2.5f : 1.7f), all = turns * product;
      float time = pt > all ? pt : all;
      if (own) time += 2.0f;
      if (time < best_time) {
        best_time = time;
        best = SplitPlan{S, blocks, own != 0};
      }
    }
  }
  return best;
}

cudaError_t launch_adapter_small(const AdapterProjHost& h, const int32_t* ids, const uint16_t* x, const uint16_t* A,
                                 const uint16_t* B, void* low, uint16_t* y, int num_sms, cudaStream_t stream) {
  const int items = h.T * ((h.r + 15) / 16);
  if (adapter_gemv_serves(h.T, h.K, h.N)) {
    const int kq = adapter_gemv_shares(h.T, h.r, h.N);
    const GemvParams p{ids, x,   h.nf4, h.absmax, A,   B,   h.scale, static_cast<float*>(low), y, h.err, h.timeout_ns,
                       h.T, h.K, h.N,   h.n,      h.r, kq,  items * kq};
    LaunchScope scope("adapter_gemv", stream);
    const int units = (h.N + 15) / 16, grid = p.p_blocks + (units < kPlaces ? units : kPlaces);
    return launch_following(h.T <= kTokenTile ? adapter_gemv_kernel<1> : adapter_gemv_kernel<2>, grid, kThreads, 0, 0,
                            stream, p);
  }
  const int NT = (h.T + 15) / 16 * 16, tiles = (h.N + ads::BM - 1) / ads::BM, chunks = h.K / ads::BK;
  const SplitPlan plan = split_plan(h, NT, tiles, chunks);
  const int S = plan.S, p_blocks = plan.own ? 0 : plan.p_blocks;
  CUtensorMap mx;
  cudaError_t err = map_bf16_2d(&mx, x, h.K, h.T, 64, (uint32_t)NT, CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  const int ring = ads::ring_bytes(NT, S), smem = ring + ads::kBarBytes + ads::kListBytes + 1024;
  const SplitParams p{h.nf4, h.absmax, x,   A,  B,   h.scale, static_cast<uint16_t*>(low), ids, y,    h.err, h.timeout_ns,
                      h.T,   NT,       h.K, h.N, h.n, h.r,    ring,                        p_blocks};
  if (plan.own) {
    LaunchScope scope("adapter_low_rank", stream);
    // an SM splits its memory for one kernel's blocks as for the other's, or they would not share it
    cudaError_t e = cudaFuncSetAttribute(adapter_low_rank_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if ((e = launch_following(adapter_low_rank_kernel, plan.p_blocks, kThreads, 0, 0, stream, p)) != cudaSuccess)
      return e;
  }
  LaunchScope scope("adapter_split", stream);
  auto run = [&](auto kernel) -> cudaError_t {
    // the same limit in every call: calls of several host threads may meet here
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ads::kMaxSmem);
    if (e != cudaSuccess) return e;
    return launch_following(kernel, p_blocks + tiles * S, ads::kThreadsSplit, smem, S, stream, mx, p);
  };
  if (h.r > 32)
    return S == 1   ? run(adapter_split_kernel<1, true>)
           : S == 2 ? run(adapter_split_kernel<2, true>)
           : S == 4 ? run(adapter_split_kernel<4, true>)
                    : run(adapter_split_kernel<8, true>);
  return S == 1   ? run(adapter_split_kernel<1, false>)
         : S == 2 ? run(adapter_split_kernel<2, false>)
         : S == 4 ? run(adapter_split_kernel<4, false>)
                  : run(adapter_split_kernel<8, false>);
}

}  // namespace e4b
