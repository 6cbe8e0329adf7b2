// Small batches of the NF4 projection with adapters of many requests.
//
//   adapter_small_proj_kernel: p[t] = bf16(s[a] A[a] x[t]) for up to 256 tokens;
//   adapter_gemv_kernel:       y[t] = W x[t] + B[a] p[t] for up to 16 tokens;
//   adapter_split_kernel:      the same for up to 256 tokens.
//
// What bounds them: reading the matrix (4.5 bits a weight) and each named
// adapter once, and the latency of two dependent launches.  The second launch
// starts while the first still runs (programmatic dependent launch), streams
// the matrix, and waits for p only before its epilogue.
//
// Up to 16 tokens the products run on warp matrix instructions (m16n8k16):
// there is nothing for a 128-row UMMA tile to amortise its set-up over.  Above,
// reading x again for every 16 rows of W would cost more than W itself, and a
// UMMA takes 128 rows of W (decoded into tensor memory) against all tokens at
// once, K split over a cluster whose partial sums meet through distributed
// shared memory.
//
// The sum over k may be taken in any order that both operands share, so in the
// warp products a lane takes 16 (x: 64) consecutive bytes of its row, and the
// elements it holds are declared to be the ones the instruction expects of it.
#include <math.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokenTile = 8;

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// D (16 x 8) += A (16 x 16) B (16 x 8), bf16 inputs, float32 sums.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg16(const void* p, bool ok) {
  return ok ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}

// ----------------------------------------------------------------------------
// p for up to kAdapterSmallTokens tokens
// ----------------------------------------------------------------------------
// A work item is (tile of up to eight tokens of one adapter, 16 of the r
// ranks): the block's warps split K, lanes read A and x straight from global
// memory, and the partial sums meet in shared memory.  GROUPED: every block
// first groups the tokens by adapter, in token order, so that all blocks find
// the same tiles (warp matches and counts in shared memory), and block 0
// leaves the tiles to the base product.  Otherwise (few
// tokens) every token is a tile of its own: grouping would cost its five block
// barriers to save reads of an adapter that L2 holds anyway.
struct SmallProjParams {
  const int32_t* ids;
  const uint16_t* x;
  const uint16_t* A;
  const float* scale;
  uint16_t* p;
  int32_t* list;  // AdapterTiles, or nullptr
  int T, K, n, r;
};

template <bool GROUPED>
__global__ void __launch_bounds__(kThreads) adapter_small_proj_kernel(const SmallProjParams p) {
  constexpr int kMax = GROUPED ? kAdapterSmallTokens : 1;
  constexpr int kCols = E4B_MAX_ADAPTERS + 16;
  static_assert(kAdapterSmallTokens == kThreads && E4B_MAX_ADAPTERS == 4 * kThreads, "one token, four adapters a thread");
  __shared__ __align__(16) uint8_t wcnt[GROUPED ? kWarps * kCols : 16];  // tokens of an adapter in a warp
  __shared__ int16_t first[GROUPED ? E4B_MAX_ADAPTERS : 1];              // an adapter's first tile
  __shared__ int16_t tile_tok[kMax * kTokenTile];          // -1: none
  __shared__ int16_t tile_ad[kMax];
  __shared__ float red[kWarps][16][kTokenTile + 1];
  __shared__ int wsum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  int n_tiles = p.T;
  if constexpr (GROUPED) {
    for (int i = tid; i < kWarps * kCols / 16; i += kThreads) reinterpret_cast<uint4*>(wcnt)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    // thread t's token: its rank among its adapter's, in token order (every block finds the same tiles)
    int ad = -1;
    if (tid < p.T) {
      const uint32_t a = (uint32_t)__ldg(p.ids + tid);
      ad = a < (uint32_t)p.n ? (int)a : p.n;
    }
    const uint32_t same = __match_any_sync(kFull, ad);
    int pos = __popc(same & ((1u << lane) - 1));
    if (ad >= 0 && pos == 0) wcnt[warp * kCols + ad] = (uint8_t)__popc(same);
    __syncthreads();
    if (ad >= 0)
      for (int w = 0; w < warp; ++w) pos += wcnt[w * kCols + ad];
    // exclusive prefix of the adapters' tiles; thread tid owns adapters 4 tid ..
    constexpr int kAds = E4B_MAX_ADAPTERS / kThreads;
    int tiles[kAds] = {}, sum = 0, none = 0;
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c4 = *reinterpret_cast<const uint32_t*>(wcnt + w * kCols + tid * kAds);
#pragma unroll
      for (int i = 0; i < kAds; ++i) tiles[i] += (c4 >> (8 * i)) & 0xffu;
      none += wcnt[w * kCols + p.n];
    }
#pragma unroll
    for (int i = 0; i < kAds; ++i) {
      tiles[i] = tid * kAds + i < p.n ? (tiles[i] + kTokenTile - 1) / kTokenTile : 0;
      sum += tiles[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int base = incl - sum;
    n_tiles = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) base += wsum[w];
      n_tiles += wsum[w];
    }
#pragma unroll
    for (int i = 0; i < kAds; ++i) {
      const int a = tid * kAds + i;
      if (a < p.n) first[a] = (int16_t)base;
      for (int j = 0; j < tiles[i]; ++j) tile_ad[base + j] = (int16_t)a;
      base += tiles[i];
    }
    const int all_tiles = n_tiles + (none + kTokenTile - 1) / kTokenTile;
    for (int i = n_tiles + tid; i < all_tiles; i += kThreads) tile_ad[i] = (int16_t)p.n;
    for (int i = tid; i < all_tiles * kTokenTile; i += kThreads) tile_tok[i] = -1;
    __syncthreads();
    if (ad >= 0) tile_tok[(ad < p.n ? first[ad] : n_tiles) * kTokenTile + pos] = (int16_t)tid;
    __syncthreads();
    if (blockIdx.x == 0) {
      if (tid == 0) p.list[0] = all_tiles;
      for (int i = tid; i < all_tiles; i += kThreads) p.list[kAdapterListAd + i] = tile_ad[i];
      for (int i = tid; i < all_tiles * kTokenTile; i += kThreads) p.list[kAdapterListTok + i] = tile_tok[i];
    }
  }

  const int g = lane >> 2, q = lane & 3;
  const int slices = (p.r + 15) / 16;
  for (int item = blockIdx.x; item < n_tiles * slices; item += gridDim.x) {
    const int tile = item / slices, j0 = (item - tile * slices) * 16;
    int a, t;
    if constexpr (GROUPED) {
      a = tile_ad[tile];
      t = tile_tok[tile * kTokenTile + g];
    } else {
      a = __ldg(p.ids + tile);
      t = g == 0 ? tile : -1;
      if ((uint32_t)a >= (uint32_t)p.n) continue;  // the whole block
    }
    const bool tok = t >= 0, lo = j0 + g < p.r, hi = j0 + g + 8 < p.r;
    const uint16_t* xr = p.x + (tok ? (size_t)t * p.K : 0) + 8 * q;
    const uint16_t* a0 = p.A + ((size_t)a * p.r + (lo ? j0 + g : 0)) * p.K + 8 * q;
    const uint16_t* a1 = p.A + ((size_t)a * p.r + (hi ? j0 + g + 8 : 0)) * p.K + 8 * q;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // 32 values of k a step: lane q of a row holds 8 of them, two instructions' worth
#pragma unroll 8
    for (int k = warp * 32; k < p.K; k += kWarps * 32) {
      const uint4 w0 = ldg16(a0 + k, lo), w1 = ldg16(a1 + k, hi), xv = ldg16(xr + k, tok);
      mma_bf16(acc, w0.x, w1.x, w0.y, w1.y, xv.x, xv.y);
      mma_bf16(acc, w0.z, w1.z, w0.w, w1.w, xv.z, xv.w);
    }
    red[warp][g][2 * q] = acc[0];
    red[warp][g][2 * q + 1] = acc[1];
    red[warp][g + 8][2 * q] = acc[2];
    red[warp][g + 8][2 * q + 1] = acc[3];
    __syncthreads();
    if (tid < 16 * kTokenTile) {
      const int j = tid & 15, c = tid >> 4;
      const int to = GROUPED ? tile_tok[tile * kTokenTile + c] : (c == 0 ? tile : -1);
      if (to >= 0 && j0 + j < p.r) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += red[w][j][c];
        const __nv_bfloat16 b = __float2bfloat16_rn(__ldg(p.scale + a) * v);
        p.p[(size_t)to * p.r + j0 + j] = *reinterpret_cast<const uint16_t*>(&b);
      }
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------------------------
// y for up to 16 tokens: 16 rows of W a block, K split over its warps
// ----------------------------------------------------------------------------
struct GemvParams {
  const int32_t* ids;
  const uint16_t* x;
  const uint8_t* nf4;
  const float* absmax;
  const uint16_t* B;
  const uint16_t* p;
  uint16_t* y;
  int T, K, N, n, r;
};

template <int NT>  // tiles of 8 tokens
__global__ void __launch_bounds__(kThreads, 2) adapter_gemv_kernel(const GemvParams p) {
  __shared__ float red[kWarps][8 * NT][17];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16;
  const bool lo = n0 + g < p.N, hi = n0 + g + 8 < p.N;
  const size_t r0 = lo ? n0 + g : 0, r1 = hi ? n0 + g + 8 : 0;
  const uint8_t* c0 = p.nf4 + r0 * (p.K / 2) + 16 * q;
  const uint8_t* c1 = p.nf4 + r1 * (p.K / 2) + 16 * q;
  const float* s0 = p.absmax + r0 * (p.K / 64) + (q >> 1);
  const float* s1 = p.absmax + r1 * (p.K / 64) + (q >> 1);
  const uint16_t* xr[NT];
  bool tok[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    tok[i] = 8 * i + g < p.T;
    xr[i] = p.x + (tok[i] ? (size_t)(8 * i + g) * p.K : 0) + 32 * q;
  }
  const Nf4Shift ks = nf4_shift_consts();
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  // A step is 128 values of k: 32 a lane, inside one block of 64.  The codes of four steps are in flight.
  const int steps = (p.K + 127) / 128;
  constexpr int kAhead = 4;
  for (int b0 = warp; b0 < steps; b0 += kWarps * kAhead) {
    uint4 w0[kAhead], w1[kAhead];
    float m0[kAhead], m1[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int b = b0 + i * kWarps;
      const bool in = b * 128 + 32 * q < p.K;  // K is a multiple of 64: the last step may be half
      w0[i] = ldg16(c0 + (size_t)b * 64, in && lo);
      w1[i] = ldg16(c1 + (size_t)b * 64, in && hi);
      m0[i] = in && lo ? __ldg(s0 + 2 * b) : 0.0f;
      m1[i] = in && hi ? __ldg(s1 + 2 * b) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int b = b0 + i * kWarps;
      if (b >= steps) break;
      const bool in = b * 128 + 32 * q < p.K;
      uint4 xv[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) xv[j][c] = ldg16(xr[j] + b * 128 + 8 * c, in && tok[j]);
      const Nf4Planes p0 = nf4_block_planes(m0[i]), p1 = nf4_block_planes(m1[i]);
      const uint32_t cw0[4] = {w0[i].x, w0[i].y, w0[i].z, w0[i].w}, cw1[4] = {w1[i].x, w1[i].y, w1[i].z, w1[i].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t d0[4], d1[4];
        nf4_decode_word(cw0[c], p0, ks, d0);
        nf4_decode_word(cw1[c], p1, ks, d1);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_bf16(acc[j], d0[0], d1[0], d0[1], d1[1], xv[j][c].x, xv[j][c].y);
          mma_bf16(acc[j], d0[2], d1[2], d0[3], d1[3], xv[j][c].z, xv[j][c].w);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    red[warp][8 * i + 2 * q][g] = acc[i][0];
    red[warp][8 * i + 2 * q + 1][g] = acc[i][1];
    red[warp][8 * i + 2 * q][g + 8] = acc[i][2];
    red[warp][8 * i + 2 * q + 1][g + 8] = acc[i][3];
  }
  // One output a thread: its adapter's row of B is fetched before p is waited for.
  const int t = tid >> 4, row = tid & 15;
  const bool mine = t < p.T && n0 + row < p.N;
  uint32_t a = 0xffffffffu;
  uint4 bw[E4B_MAX_RANK / 8];
  if (mine) a = (uint32_t)__ldg(p.ids + t);
  const bool adapted = mine && a < (uint32_t)p.n;
#pragma unroll
  for (int j = 0; j < E4B_MAX_RANK / 8; ++j)
    bw[j] = ldg16(p.B + ((size_t)(adapted ? a : 0) * p.N + (mine ? n0 + row : 0)) * p.r + 8 * j,
                  adapted && 8 * j < p.r);
  __syncthreads();
  grid_wait();
  if (mine) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][t][row];
    if (adapted) {
      const uint4* pr = reinterpret_cast<const uint4*>(p.p + (size_t)t * p.r);
#pragma unroll
      for (int j = 0; j < E4B_MAX_RANK / 8; ++j) {
        if (8 * j >= p.r) break;
        const uint4 pv = __ldcg(pr + j);
        const uint32_t b4[4] = {bw[j].x, bw[j].y, bw[j].z, bw[j].w}, p4[4] = {pv.x, pv.y, pv.z, pv.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          v = fmaf(bf16lo_to_f32(b4[c]), bf16lo_to_f32(p4[c]), v);
          v = fmaf(bf16hi_to_f32(b4[c]), bf16hi_to_f32(p4[c]), v);
        }
      }
    }
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    p.y[(size_t)t * p.N + n0 + row] = *reinterpret_cast<const uint16_t*>(&h);
  }
}

// ----------------------------------------------------------------------------
// y for up to 256 tokens: 128 rows of W x all tokens x a share of K per block
// ----------------------------------------------------------------------------
// Warp 0 loads x tiles (TMA), warp 1 owns tensor memory and issues the UMMAs,
// warps 4-15 are three decode teams that take the k-chunks round robin: a
// thread owns a row of W, reads 32 bytes of codes and a scale a chunk straight
// into registers two of its chunks ahead, and writes the decoded row to the A
// buffer in tensor memory.  Then every block's partial sums go to its shared
// memory (over the x tiles), the cluster's blocks each add up 128 / S rows over
// the S shares of K, and the adapters' part is added in the fragment layout of
// the warp instruction, tile by tile of eight tokens of one adapter, so that
// no adapter's values meet another's tokens.
namespace ads {
constexpr int BM = 128, BK = 64;
constexpr int kXStages = 4, kTeams = 3, kABufs = 2 * kTeams, kACols = BK / 2;
constexpr int kThreadsSplit = 512;
constexpr int kAOff = 256;             // TMEM columns: accumulator [0, 256), A buffers behind
constexpr int kPitch = BM + 4;         // floats of a token's partial sums (no bank conflicts in fragment reads)
constexpr int kTmemCols = 512;
inline int ring_bytes(int nt) {
  const int x = kXStages * nt * BK * 2, part = nt * kPitch * 4;
  return ((x > part ? x : part) + 1023) / 1024 * 1024;
}
static_assert(kAOff + kABufs * kACols <= kTmemCols, "TMEM budget");
}  // namespace ads

struct SplitParams {
  const uint8_t* nf4;
  const float* absmax;
  const uint16_t* B;
  const uint16_t* p;
  const int32_t* list;
  uint16_t* y;
  DeviceError* err;
  long long timeout_ns;
  int T, NT, K, N, n, r, S;  // NT: T rounded up to 16
  int ring;                  // bytes of the x ring / partial sums
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(ads::kThreadsSplit, 1)
    adapter_split_kernel(const __grid_constant__ CUtensorMap map_x, const SplitParams p) {
  using namespace ads;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ring);
  uint64_t* x_full = bars;                  // [kXStages]
  uint64_t* x_empty = x_full + kXStages;    // [kXStages]
  uint64_t* a_ready = x_empty + kXStages;   // [kABufs] a team's decoded chunk is in tensor memory (4 warps)
  uint64_t* a_empty = a_ready + kABufs;     // [kABufs]
  uint64_t* accfull = a_empty + kABufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accfull + 1);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(accfull + 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)(blockIdx.x % p.S), n0 = (int)(blockIdx.x / p.S) * BM;
  const int chunks = p.K / BK;
  const int k_lo = rank * chunks / p.S, nc = (rank + 1) * chunks / p.S - k_lo;
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
  const int x_bytes = p.NT * BK * 2;

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
    // partial sums to shared memory, [token][row]; the UMMAs have read the last x tile.  Team by team 16 columns.
    if (__all_sync(kFull, mbar_wait(accfull, 0, ctl, p.err, p.timeout_ns, 631))) {
      tc_fence_after();
      float* part = reinterpret_cast<float*>(smem) + 32 * (warp & 3) + lane;
      for (int c = 16 * team; c < p.NT; c += 16 * kTeams) {
        float v[16];
        tmem_ld16(tmem + c + ((uint32_t)(32 * (warp & 3)) << 16), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kPitch] = v[i];
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync();  // every block's partial sums are in place
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  grid_wait();  // p and the token tiles
  {
    // This block's rows: 128 / S of the 128, in groups of 16; item = (group, tile of 8 tokens).
    const int rows = BM / p.S, groups = rows / 16, g = lane >> 2, q = lane & 3;
    const int n_tiles = __ldcg(p.list);
    const uint32_t part_u = smem_u32(smem);
    for (int item = warp; item < n_tiles * groups; item += kThreadsSplit / 32) {
      const int tile = item / groups, grp = item - tile * groups;
      const int lrow = rank * rows + 16 * grp, row = n0 + lrow;
      if (row >= p.N) continue;  // the whole warp (N is a multiple of 8: the second half may still be outside)
      const int a = __ldcg(p.list + kAdapterListAd + tile);
      const int* toks = p.list + kAdapterListTok + tile * kTokenTile;
      const int tg = __ldcg(toks + g);                                            // fragment B column
      const int t0 = __ldcg(toks + 2 * q), t1 = __ldcg(toks + 2 * q + 1);         // fragment D columns
      const bool hi = row + 8 < p.N;
      uint4 b0[2], b1[2], pv[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int j = 32 * c + 8 * q;
        const bool go = a < p.n && j < p.r && row + g < p.N;
        b0[c] = ldg16(p.B + ((size_t)(go ? a : 0) * p.N + (go ? row + g : 0)) * p.r + (go ? j : 0), go);
        b1[c] = ldg16(p.B + ((size_t)(go ? a : 0) * p.N + (go && hi ? row + g + 8 : 0)) * p.r + (go ? j : 0), go && hi);
        pv[c] = make_uint4(0, 0, 0, 0);
        if (go && tg >= 0) pv[c] = __ldcg(reinterpret_cast<const uint4*>(p.p + (size_t)tg * p.r + j));
      }
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t o0 = (uint32_t)(((t0 < 0 ? 0 : t0) * kPitch + lrow + g) * 4);
      const uint32_t o1 = (uint32_t)(((t1 < 0 ? 0 : t1) * kPitch + lrow + g) * 4);
      for (int s = 0; s < p.S; ++s) {  // the shares of K, in order
        const uint32_t base = mapa_shared(part_u, (uint32_t)s);
        d[0] += ld_cluster_f32(base + o0);
        d[1] += ld_cluster_f32(base + o1);
        d[2] += ld_cluster_f32(base + o0 + 32);
        d[3] += ld_cluster_f32(base + o1 + 32);
      }
      if (a < p.n) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (32 * c < p.r) {
            mma_bf16(d, b0[c].x, b1[c].x, b0[c].y, b1[c].y, pv[c].x, pv[c].y);
            mma_bf16(d, b0[c].z, b1[c].z, b0[c].w, b1[c].w, pv[c].z, pv[c].w);
          }
      }
      auto put = [&](int t, int r, float f) {
        const __nv_bfloat16 h = __float2bfloat16_rn(f);
        if (t >= 0 && r < p.N) p.y[(size_t)t * p.N + r] = *reinterpret_cast<const uint16_t*>(&h);
      };
      put(t0, row + g, d[0]);
      put(t1, row + g, d[1]);
      put(t0, row + g + 8, d[2]);
      put(t1, row + g + 8, d[3]);
    }
  }
  __syncwarp();
  cluster_sync();  // no block's shared memory goes away while another reads it
}

// Launches `kernel` so that it may start before the launch ahead of it in the stream has finished (it calls
// griddepcontrol.wait before it reads what that launch wrote).
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), int grid, int threads, int smem, int cluster,
                             cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_adapter_small(const AdapterProjHost& h, const int32_t* ids, const uint16_t* x, const uint16_t* A,
                                 const uint16_t* B, uint16_t* low, int32_t* list, uint16_t* y, int num_sms,
                                 cudaStream_t stream) {
  const bool few = h.T <= kAdapterGemvTokens;
  {
    const SmallProjParams p{ids, x, A, h.scale, low, list, h.T, h.K, h.n, h.r};
    // at most T tiles, and at most T / 8 full ones with one more an adapter
    const int tiles = few || h.T < h.T / kTokenTile + h.n ? h.T : h.T / kTokenTile + h.n;
    const int items = tiles * ((h.r + 15) / 16);
    const int grid = items < 4 * num_sms ? items : 4 * num_sms;
    LaunchScope scope("adapter_small_proj", stream);
    if (few)
      adapter_small_proj_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    else
      adapter_small_proj_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  if (few) {
    const GemvParams p{ids, x, h.nf4, h.absmax, B, low, y, h.T, h.K, h.N, h.n, h.r};
    LaunchScope scope("adapter_gemv", stream);
    const int grid = (h.N + 15) / 16;
    return h.T <= kTokenTile ? launch_dependent(adapter_gemv_kernel<1>, grid, kThreads, 0, 0, stream, p)
                             : launch_dependent(adapter_gemv_kernel<2>, grid, kThreads, 0, 0, stream, p);
  }
  const int NT = (h.T + 15) / 16 * 16, tiles = (h.N + ads::BM - 1) / ads::BM, chunks = h.K / ads::BK;
  // K is split while the blocks fit the GPU at once and every block keeps two chunks.
  int S = 1;
  while (S < 8 && 2 * S * tiles <= num_sms && chunks >= 4 * S) S *= 2;
  CUtensorMap mx;
  cudaError_t err = map_bf16_2d(&mx, x, h.K, h.T, 64, (uint32_t)NT, CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  const int ring = ads::ring_bytes(NT), smem = ring + 1024 + 1024;
  const SplitParams p{h.nf4, h.absmax, B, low, list, y, h.err, h.timeout_ns, h.T, NT, h.K, h.N, h.n, h.r, S, ring};
  if ((err = cudaFuncSetAttribute(adapter_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
      cudaSuccess)
    return err;
  LaunchScope scope("adapter_split", stream);
  return launch_dependent(adapter_split_kernel, tiles * S, ads::kThreadsSplit, smem, S, stream, mx, p);
}

}  // namespace e4b
