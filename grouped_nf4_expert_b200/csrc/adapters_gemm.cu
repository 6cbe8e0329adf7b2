// Large batches of the NF4 projection with adapters of many requests, on the
// 5th-generation tensor cores:
//
//  * adapter_fwd_kernel, adapter_dgrad_kernel: persistent CTA pairs, 256 token
//    rows (forward: up to 384) x 256 outputs per work unit (cta_group::2 UMMAs): the base product with
//    the NF4 matrix decoded on the way, then one K = r step per adapter with rows
//    in the tile, written to that adapter's rows only.
//  * adapter_proj_kernel: p = s x A^T and q = s dY B, 128 rows of one adapter
//    at a time.
//  * adapter_wgrad_kernel: dA = q^T x and dB = dY^T p, K = the rows of one
//    adapter.
//
// Rows are the tokens sorted by adapter; every adapter's rows start at a
// multiple of 32: the column granule of a pair UMMA (forward), and two K steps of
// a UMMA, so that the gradient products never multiply two adapters' rows.  The
// projection kernel gathers the token rows (cp.async, 16 bytes a lane) and stores
// them in row order in passing, for the base product to load as plain tiles.  TMA
// gathers by row index (tile::gather4) were measured instead: about 77 cycles for
// every four rows of 128 bytes, 5 times the time of the UMMAs they feed (T =
// 16384, K = 4096, N = 14336, both with one issuing warp and relays: 4204 us
// against 1960 us with the copy).
//
// The adapters of a tile share its accumulator: each K = r step is issued at the
// adapter's own accumulator columns (forward) or names the TMEM lanes it must not
// write (input gradient: the disable-output-lane operand), so the rows need not
// be split into tiles by adapter, and nothing an adapter or a token holds reaches
// another request's rows.
#include <math.h>

#include "e4b_device.cuh"
#include "e4b_internal.h"
#include "launch.cuh"

namespace e4b {

namespace {

constexpr uint32_t kFull = 0xffffffffu;

// The pair UMMA with output lanes disabled: bit i of the 256-bit mask keeps row i of the accumulator as it is.
__device__ __forceinline__ void umma_bf16_2sm_masked(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                     const uint32_t (&off)[8]) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, 1, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]), "r"(off[5]),
      "r"(off[6]), "r"(off[7])
      : "memory");
}

// The pair UMMA with the M operand in tensor memory (each CTA's 128 rows in its own).
__device__ __forceinline__ void umma_bf16_2sm_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// After a wait ran out, time for copies in flight to land before the shared memory goes away.
constexpr uint64_t kLandNs = 1000000;

// The adapters of a unit of up to 32 kMost rows from row0 on, one run of rows [lo, hi) (relative to row0) at a time: the
// adapter of every 32 rows is in `granules` (n for the tokens without one), and every adapter starts such a granule.
// All of them are read at once, when the unit starts.
template <int kMost>
struct AdapterRun {
  int id[kMost];
  int n, granule = 0;
  int lo = 0, hi = 0, adapter = -1;
  __device__ __forceinline__ AdapterRun(const int32_t* granules, int row0, int rows_used, int rows, int n_) : n(n_) {
    rows = min(rows, rows_used - row0);
#pragma unroll
    for (int i = 0; i < kMost; ++i)
      id[i] = i * kAdapterRowAlign < rows ? __ldg(granules + row0 / kAdapterRowAlign + i) : n;
  }
  __device__ __forceinline__ int at(int i) const {
    int a = n;
#pragma unroll
    for (int j = 0; j < kMost; ++j)
      if (j == i) a = id[j];
    return a;
  }
  __device__ __forceinline__ bool next() {
    adapter = at(granule);
    if (adapter >= n) return false;  // the rest has none
    lo = granule * kAdapterRowAlign;
    do {
      ++granule;
    } while (at(granule) == adapter);
    hi = granule * kAdapterRowAlign;
    return true;
  }
};

// TMA loads whose completion is counted on a barrier of either CTA of the pair (a cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                                 int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Mask word w (rows 32 w ..) with the bits outside rows [lo, hi) set.
__device__ __forceinline__ uint32_t rows_off(int lo, int hi, int w) {
  const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
  const uint32_t below_b = b == 32 ? kFull : (1u << b) - 1;
  const uint32_t below_a = a == 32 ? kFull : (1u << a) - 1;
  return ~(below_b & ~below_a);
}

// Shares of a 128 x r_pad accumulator over a cluster of S blocks that split its reduction: block b owns rows
// [128 b / S, 128 (b + 1) / S).  push_share: an epilogue warp stores its 32 TMEM lanes (zeros unless `live`)
// into the owners' shared memory, [share][column][row]: a warp's store is one run of rows.  (Rows first, its 32
// lanes' stores went out as 32 packets, 8 us a block of 64 columns.)  sum_share adds four columns of an owned row
// in share order.
constexpr int kSharePad = 4;
constexpr int share_bytes(int r_pad, int S) { return r_pad * (128 + S * kSharePad) * 4; }
__device__ __forceinline__ void push_share(uint8_t* smem, uint32_t tmem, int quarter, int lane, int S, int rank,
                                           int r_pad, bool live) {
  const int rows = 128 / S, row = 32 * quarter + lane, pitch = rows + kSharePad;
  const uint32_t to =
      mapa_shared(smem_u32(smem) + (uint32_t)((rank * r_pad * pitch + row % rows) * 4), (uint32_t)(row / rows));
  for (int j = 0; j < r_pad; j += 16) {
    float v[16];
    if (live) {
      tmem_ld16(tmem + j + ((uint32_t)(32 * quarter) << 16), v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + (uint32_t)((j + i) * pitch * 4)), "f"(v[i])
                   : "memory");
  }
}
__device__ __forceinline__ float4 sum_share(const uint8_t* smem, int S, int row, int j, int r_pad) {
  const int pitch = 128 / S + kSharePad;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int s = 0; s < S; ++s) {
    const float* at = reinterpret_cast<const float*>(smem) + (s * r_pad + j) * pitch + row;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += at[i * pitch];
  }
  return make_float4(v[0], v[1], v[2], v[3]);
}

// Waits (with the limit) until the copies this role issued have landed, before its shared memory goes away.
__device__ __forceinline__ void let_land(uint64_t* bars, int n, uint32_t issued, uint32_t last_par,
                                         long long timeout_ns) {
  for (int i = 0; i < n; ++i)
    if (issued & (1u << i)) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&bars[i], (last_par >> i) & 1u) && (long long)(globaltimer_ns() - t0) < timeout_ns) {
      }
    }
}

}  // namespace

// =============================================================================
// Forward: y[t] = W x[t] + B[a] p[t], W as the M operand
// =============================================================================
// A unit is 256 rows of W (128 a CTA of the pair) x up to 256 token rows, or 384
// where one turn of the pairs does then (a multiple of 32, chosen so that the units
// fill the pairs evenly).  A thread of
// the decode groups owns a row of W: it decodes 64 weights of a k-chunk into
// registers and writes them to tensor memory, where the UMMAs read their M
// operand.  Written to shared memory instead (as the expert block's tiles are,
// and the input gradient's below), the decoded tile costs 16 KB of writes and 16
// KB of operand reads a chunk on top of the token rows' 32 KB: more
// shared-memory time than the chunk's 512 tensor cycles.
//
// The accumulator is in parts of 128 token rows (the last one may be smaller), in
// three TMEM slots used in turn, and each part has an issuing warp of its own: while
// the epilogue empties the first part of a unit of two, the next unit's first part
// fills, and the second follows once its slot is free.  (One warp handing in two
// parts' products took 720 cycles a chunk, against 512 in the tensor pipe: its
// instruction stream, not the operands, was the limit.)  Units of three parts have
// no slot to spare and are used for a single turn: 1111 tokens, 2048 -> 4096, the
// whole call with 64 units of 384 rows 40.7 us, with 128 of 160 45.4 us.  Token rows
// are accumulator columns, so an adapter's K = r product is issued at its own columns:
// adapters' rows start at multiples of 32, the column granule of a pair UMMA.
//
// The issuers see both CTAs' operands on barriers of the even CTA: the odd CTA's
// TMA loads count their bytes there, and its decode warps signal with a 4-byte
// st.async each.  (A relay warp that waited for a CTA's operands and passed one
// signal on took about 690 cycles a chunk: beside four decode warps on its
// scheduler, every instruction of it waits for a turn.)
//
// A chunk bounds it, the tensor pipe's part and the decode beside it: 840 cycles with
// 256 rows (512 in the tensor pipe), 680 with 128 and less.  8192 tokens, 2048 -> 2048:
// 72 us, 960 TFLOP/s, tensor pipe 52% active: 224-row units in four full turns, 448 of
// a chunk's 823 cycles; 16384 tokens, 4096 -> 14336: 1.08 PFLOP/s over the whole call.
//
// Roles per CTA: warp 0 codes, warp 1 TMEM owner and (even CTA) issuer of the
// first parts, warp 2 (even CTA) issuer of the second parts, warp 3 token rows and
// low-rank operands, warps 4-19 four decode groups taking the chunks round robin,
// warps 20-23 epilogue (32 rows of W each), warp 24 issuer of third parts.
namespace adf {
constexpr int BM = 128, BK = 64;
constexpr int kHalf = 128;                    // token rows of an accumulator part
constexpr int kPartBytes = kHalf / 2 * BK * 2;  // a CTA's 64 token rows of a part and chunk
constexpr int slot_bytes(int parts) { return parts * kPartBytes; }
constexpr int slots(int parts) { return parts > 2 ? 5 : 8; }  // token-row ring
constexpr int kGroups = 4, kGroupWarps = 4;
constexpr int kSlots = 3;                     // accumulator parts
constexpr int kAOff = kSlots * kHalf;         // TMEM: the parts, then one decoded chunk (32 columns) a group
constexpr int RAW_STAGES = 2 * kGroups, RAW_BYTES = BM * BK / 2;
constexpr int RAW_OFF = slots(2) * slot_bytes(2);
constexpr int EPI_OFF = RAW_OFF + RAW_STAGES * RAW_BYTES;
constexpr int kEpiPitch = 80;                 // bytes of a token's 32 outputs of a warp, padded
constexpr int kEpiWarpBytes = 32 * kEpiPitch;
constexpr int BAR_OFF = EPI_OFF + 4 * kEpiWarpBytes;
constexpr int SMEM_BYTES = BAR_OFF + 1024 + 1024;
constexpr int kEpiWarp0 = 4 + kGroups * kGroupWarps;
constexpr int kThirdWarp = kEpiWarp0 + 4;
constexpr int threads(int parts) { return 32 * (kThirdWarp + (parts > 2)); }
constexpr int kTmemCols = 512;
static_assert(kAOff + kGroups * BK / 2 <= kTmemCols, "TMEM budget");
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
static_assert(slots(3) * slot_bytes(3) <= RAW_OFF, "the ring of three parts fits");
static_assert(BM * E4B_MAX_RANK * 2 <= slot_bytes(2) && 64 * E4B_MAX_RANK * 2 <= kPartBytes, "low-rank operands fit");
}  // namespace adf

struct AdapterFwdParams {
  const float* absmax;
  const int32_t* order;
  const int32_t* steps;
  uint16_t* out;
  DeviceError* err;
  long long timeout_ns;
  int K, N, T, n_adapters, r_pad, n_mt;
  int n[3];  // token rows of a unit's parts, multiples of 32: 128 where another part follows, 0 where there is none
};

// Rows [lo, hi) of a run in part i of its unit (n rows from 128 i on), relative to the part.
template <typename Run>
__device__ __forceinline__ int2 part_range(const Run& run, int i, int n) {
  return make_int2(min(max(run.lo - adf::kHalf * i, 0), n), min(max(run.hi - adf::kHalf * i, 0), n));
}

template <int PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(adf::threads(PARTS), 1)
    adapter_fwd_kernel(const __grid_constant__ CUtensorMap map_x0, const __grid_constant__ CUtensorMap map_x1,
                       const __grid_constant__ CUtensorMap map_raw, const __grid_constant__ CUtensorMap map_p,
                       const __grid_constant__ CUtensorMap map_b, const AdapterFwdParams p) {
  using namespace adf;
  using Run = AdapterRun<4 * PARTS>;
  constexpr int X_BYTES = slot_bytes(PARTS), SA = slots(PARTS);
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  uint8_t* rawbuf = smem + RAW_OFF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
  uint64_t* raw_full = bars;                    // [RAW_STAGES] codes landed
  uint64_t* raw_empty = raw_full + RAW_STAGES;  // [RAW_STAGES] codes read into registers (group's 4 warps)
  uint64_t* xfull = raw_empty + RAW_STAGES;     // [SA] (even CTA) ring use landed in both CTAs
  uint64_t* xempty = xfull + SA;                // [SA] ring slot consumed by the UMMAs
  uint64_t* adone = xempty + SA;                // [kGroups] (even CTA) both CTAs' decoded chunk is in tensor memory
  uint64_t* aempty = adone + kGroups;           // [kGroups] decoded chunk consumed by the UMMAs
  uint64_t* accfull = aempty + kGroups;         // [kSlots] accumulator part complete
  uint64_t* accempty = accfull + kSlots;        // [kSlots] (even CTA) part drained in both CTAs
  uint64_t* drain = accempty + kSlots;          // [3] (even CTA) all of an issuer's UMMAs finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 3);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(drain + 4);
  uint32_t* sig = reinterpret_cast<uint32_t*>(drain + 5);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int parts = 1 + (p.n[1] > 0) + (PARTS > 2);
  if (threadIdx.x == 0) {
    for (int r = 0; r < RAW_STAGES; ++r) {
      mbar_init(&raw_full[r], 1);
      mbar_init(&raw_empty[r], kGroupWarps);
    }
    for (int s = 0; s < SA; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&xempty[s], parts);
    }
    for (int g = 0; g < kGroups; ++g) {
      mbar_init(&adone[g], kGroupWarps);
      mbar_init(&aempty[g], parts);
    }
    for (int b = 0; b < kSlots; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 8);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&drain[i], 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_2sm(tmem_slot, kTmemCols);
    tmem_relinquish_2sm();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  grid_launch_dependents();

  const int rows_used = p.steps[0], unit_rows = p.n[0] + p.n[1] + (PARTS > 2 ? p.n[2] : 0);
  const int n_units = (rows_used + unit_rows - 1) / unit_rows * p.n_mt;
  const int kchunks = p.K / BK;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int32_t* granules = p.steps + kAdapterStepsHeader;
  const bool pack = p.r_pad <= 32;  // both halves of the low-rank rows in one slot

  if (warp == 0) {
    // ------------------------------------------------ NF4 codes: 128 rows x 32 bytes a chunk (one lane)
    if (lane == 0) {
      tma_prefetch_desc(&map_raw);
      uint32_t j = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += n_pairs) {
        const int row0 = (u % p.n_mt) * 256 + (int)rank * BM;
        for (int kc = 0; kc < kchunks; ++kc, ++j) {
          const uint32_t r = j % RAW_STAGES, ph = (j / RAW_STAGES) & 1;
          if (!(ok = mbar_wait_lazy(&raw_empty[r], ph ^ 1, ctl, p.err, p.timeout_ns, 211, 64))) break;
          mbar_arrive_expect_tx(&raw_full[r], (uint32_t)RAW_BYTES);
          tma_load_2d(rawbuf + r * RAW_BYTES, &map_raw, &raw_full[r], kc * (BK / 2), row0);
          issued |= 1u << r;
          last_par = (last_par & ~(1u << r)) | (ph << r);
        }
      }
      if (!ok) let_land(raw_full, RAW_STAGES, issued, last_par, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------ token rows, then a unit's low-rank operands (one lane)
    // This CTA's rows of a part: 64 of its 128 (of an adapter's columns: half of them).  A low-rank use is
    // two slots, the adapter's 128 rows of B, then both halves of its p rows of every part, or (64 ranks) three.
    if (lane == 0) {
      tma_prefetch_desc(&map_x0);
      tma_prefetch_desc(&map_p);
      tma_prefetch_desc(&map_b);
      // Completions are counted on the even CTA's xfull, which its loader arms for both CTAs' (equal) bytes.
      const uint32_t xfull_even = mapa_shared(smem_u32(xfull), 0);
      uint32_t s = 0, ph = 0;
      auto issued_next = [&]() {
        if (++s == SA) {
          s = 0;
          ph ^= 1;
        }
      };
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += n_pairs) {
        const int w0 = (u % p.n_mt) * 256 + (int)rank * BM, t0 = u / p.n_mt * unit_rows;
        Run run(granules, t0, rows_used, unit_rows, p.n_adapters);
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!(ok = mbar_wait(&xempty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 212))) break;
          uint8_t* x = smem + s * X_BYTES;
          const uint32_t bar = xfull_even + 8 * s;
          if (rank == 0) mbar_arrive_expect_tx(&xfull[s], (uint32_t)(2 * unit_rows * BK));
          tma_load_2d_pair(x, &map_x0, bar, kc * BK, t0 + p.n[0] / 2 * (int)rank);
          if (PARTS > 2) {
            tma_load_2d_pair(x + kPartBytes, &map_x0, bar, kc * BK, t0 + kHalf + p.n[1] / 2 * (int)rank);
            tma_load_2d_pair(x + 2 * kPartBytes, &map_x1, bar, kc * BK, t0 + 2 * kHalf + p.n[2] / 2 * (int)rank);
          } else if (p.n[1]) {
            tma_load_2d_pair(x + kPartBytes, &map_x1, bar, kc * BK, t0 + kHalf + p.n[1] / 2 * (int)rank);
          }
          issued_next();
        }
        if (!ok) break;
        while (run.next()) {
          const uint32_t s1 = (s + 1 == SA) ? 0 : s + 1, ph1 = (s + 1 == SA) ? ph ^ 1 : ph;
          const uint32_t s2 = (s1 + 1 == SA) ? 0 : s1 + 1, ph2 = (s1 + 1 == SA) ? ph1 ^ 1 : ph1;
          if (!(ok = mbar_wait(&xempty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 210))) break;
          if (!(ok = mbar_wait(&xempty[s1], ph1 ^ 1, ctl, p.err, p.timeout_ns, 210))) break;
          if (!pack && !(ok = mbar_wait(&xempty[s2], ph2 ^ 1, ctl, p.err, p.timeout_ns, 210))) break;
          int rows[PARTS], first[PARTS], all = 0;  // this CTA's p rows of each part, multiples of 16
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            const int2 h = part_range(run, i, p.n[i]);
            rows[i] = (h.y - h.x) / 2;
            first[i] = t0 + kHalf * i + h.x + rows[i] * (int)rank;
            all += rows[i];
          }
          const uint32_t bar = xfull_even + 8 * s;
          if (rank == 0) {
            mbar_arrive_expect_tx(&xfull[s], (uint32_t)((BM + 2 * all) * 4 * p.r_pad));
            mbar_arrive(&xfull[s1]);
            if (!pack) mbar_arrive(&xfull[s2]);
          }
          uint8_t* b = smem + s * X_BYTES;
          tma_load_3d_pair(b, &map_b, bar, 0, w0, run.adapter);
          tma_load_3d_pair(b + 128 * p.r_pad, &map_b, bar, 0, w0 + 64, run.adapter);
          uint8_t* high = smem + s1 * X_BYTES;
          uint8_t* low = pack ? high + X_BYTES / 2 : smem + s2 * X_BYTES;
#pragma unroll
          for (int i = 0; i < PARTS; ++i)
            for (int k = 0; k < rows[i]; k += 16) {
              const int at = (64 * i + k) * 2 * p.r_pad;
              tma_load_3d_pair(high + at, &map_p, bar, 0, 0, first[i] + k);
              tma_load_3d_pair(low + at, &map_p, bar, 0, 1, first[i] + k);
            }
          issued_next();
          issued_next();
          if (!pack) issued_next();
        }
      }
      // (After a wait ran out: copies of either CTA may be in flight; they are given time to land.)
      if (!ok) {
        const uint64_t c0 = globaltimer_ns();
        while (globaltimer_ns() - c0 < kLandNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 || warp == 2 || warp == kThirdWarp) {
    // ------------------------------------------------ UMMA issuers (even CTA, one elected lane each)
    const int h = warp == kThirdWarp ? 2 : warp - 1;  // its part
    if (rank == 0 && h < parts && elect_one_sync()) {
      const int rows = h == 0 ? p.n[0] : h == 1 ? p.n[1] : p.n[2];
      const uint32_t idesc = make_idesc_bf16(256, rows, false, false);
      const uint32_t lswz = swz_for_row_bytes(2 * p.r_pad);
      const uint32_t x_u = smem_u32(smem);
      const uint64_t xdesc0 = make_sdesc(x_u + h * kPartBytes, 16, 1024, kSw128);
      uint32_t sx = 0, phx = 0, g = 0, pha = 0, hs = h;  // ring slot, decode group, accumulator part used
      bool ok = true;
      auto next_x = [&]() {
        if (++sx == SA) {
          sx = 0;
          phx ^= 1;
        }
      };
      auto wait_x = [&]() -> bool { return mbar_wait_cluster(&xfull[sx], phx, ctl, p.err, p.timeout_ns, 223); };
      for (int u = pair; u < n_units && ok; u += n_pairs, hs += parts) {
        const uint32_t slot = hs % kSlots, d = tmem + slot * kHalf;
        Run run(granules, u / p.n_mt * unit_rows, rows_used, unit_rows, p.n_adapters);
        if (!(ok = mbar_wait_cluster(&accempty[slot], ((hs / kSlots) & 1) ^ 1, ctl, p.err, p.timeout_ns, 220))) break;
        tc_fence_after();
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!(ok = wait_x())) break;
          if (!(ok = mbar_wait_cluster(&adone[g], pha, ctl, p.err, p.timeout_ns, 224))) break;
          tc_fence_after();
          const uint32_t a = tmem + kAOff + g * (BK / 2);
          const uint64_t xd = xdesc0 + (uint64_t)(sx * (X_BYTES >> 4));
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma_bf16_2sm_ta(d, a + 8 * kk, xd + 2 * kk, idesc, (kc > 0 || kk > 0) ? 1u : 0u);
          umma_commit_2sm(&xempty[sx], 0x3);
          umma_commit_2sm(&aempty[g], 0x3);
          next_x();
          if (++g == kGroups) {
            g = 0;
            pha ^= 1;
          }
        }
        if (!ok) break;
        // One K = r product per adapter, at the adapter's columns of this part.
        while (run.next()) {
          if (!(ok = wait_x())) break;
          tc_fence_after();
          const uint32_t sx1 = (sx + 1 == SA) ? 0 : sx + 1, sx2 = (sx1 + 1 == SA) ? 0 : sx1 + 1;
          const uint32_t b_u = x_u + sx * X_BYTES, part = x_u + h * 128 * p.r_pad;
          const uint32_t p_u[2] = {part + sx1 * X_BYTES, part + (pack ? sx1 * X_BYTES + X_BYTES / 2 : sx2 * X_BYTES)};
          const int2 hr = part_range(run, h, rows);
          if (hr.y > hr.x) {
            const uint32_t id = make_idesc_bf16(256, hr.y - hr.x, false, false);
            for (int ks = 0; ks < p.r_pad / 16; ++ks)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                umma_bf16_2sm(d + hr.x, make_sdesc(b_u + 32 * ks, 16, 16 * p.r_pad, lswz),
                              make_sdesc(p_u[i] + 32 * ks, 16, 16 * p.r_pad, lswz), id, 1u);
          }
          umma_commit_2sm(&xempty[sx], 0x3);
          umma_commit_2sm(&xempty[sx1], 0x3);
          if (!pack) umma_commit_2sm(&xempty[sx2], 0x3);
          next_x();
          next_x();
          if (!pack) next_x();
        }
        if (!ok) break;
        umma_commit_2sm(&accfull[slot], 0x3);
      }
      umma_commit_2sm(&drain[h], 0x1);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(&drain[h], 0) && (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < kEpiWarp0) {
    // ------------------------------------------------ NF4 decode: a row of W a thread
    const uint32_t grp = (warp - 4) >> 2;
    const uint32_t adone_even = mapa_shared(smem_u32(adone + grp), 0), sig_even = mapa_shared(smem_u32(sig), 0);
    const int t = (threadIdx.x - 128) & 127;
    const Nf4Shift ks = nf4_shift_consts();
    const uint32_t a_base = tmem + kAOff + grp * (BK / 2) + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t my_units = pair < n_units ? (uint32_t)((n_units - pair + n_pairs - 1) / n_pairs) : 0;
    const uint32_t n_chunks = my_units * (uint32_t)kchunks;
    // A cursor over this group's chunks, one ahead of the decode (for the block scales).
    int c_kc = (int)grp, c_u = pair;
    auto wrap = [&]() {
      while (c_kc >= kchunks) {
        c_kc -= kchunks;
        c_u += n_pairs;
      }
    };
    wrap();
    int c_row = (c_u % p.n_mt) * 256 + (int)rank * BM + t;
    auto block_scale = [&]() -> float {  // 0 past the end of the matrix: zero weights
      if (c_u >= n_units || c_row >= p.N) return 0.0f;
      return __ldg(p.absmax + (size_t)c_row * kchunks + c_kc);
    };
    float amax_next = block_scale();
    bool ok = true;
    for (uint32_t jj = grp; jj < n_chunks && ok; jj += kGroups) {
      const float amax = amax_next;
      const int old = c_u;
      c_kc += kGroups;
      wrap();
      if (c_u != old) c_row = (c_u % p.n_mt) * 256 + (int)rank * BM + t;
      const uint32_t r = jj % RAW_STAGES, rph = (jj / RAW_STAGES) & 1;
      ok = __all_sync(kFull, mbar_wait(&raw_full[r], rph, ctl, p.err, p.timeout_ns, 230));
      if (!ok) break;
      const uint8_t* slot = rawbuf + r * RAW_BYTES + t * 32;
      const uint4 q0 = *reinterpret_cast<const uint4*>(slot);
      const uint4 q1 = *reinterpret_cast<const uint4*>(slot + 16);
      const uint32_t codes[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      fence_proxy_async_smem();  // these reads before the next TMA write of the slot
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_empty[r]);
      amax_next = block_scale();
      const Nf4Planes pl = nf4_block_planes(amax);
      uint32_t v[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) nf4_decode_word(codes[c], pl, ks, &v[4 * c]);
      ok = __all_sync(kFull, mbar_wait(&aempty[grp], ((jj / kGroups) & 1) ^ 1, ctl, p.err, p.timeout_ns, 231));
      if (!ok) break;
      tc_fence_after();
      tmem_st32(a_base, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank)
          st_async_signal(sig_even, adone_even, 1u);
        else if ((warp & 3) == 0)
          mbar_arrive_expect_tx(&adone[grp], 4 * kGroupWarps);  // and the odd CTA's four signals
        else
          mbar_arrive(&adone[grp]);
      }
    }
  } else if (warp >= kEpiWarp0) {  // (the third issuer is taken above)
    // ------------------------------------------------ epilogue: 32 rows of W x the token rows
    // A lane holds a row of W; 32 token rows at a time pass through shared memory so that a store writes 64
    // contiguous bytes of each of eight tokens.
    const int qrt = warp & 3;
    const uint32_t accempty_even = mapa_shared(smem_u32(accempty), 0);
    uint8_t* ebuf = smem + EPI_OFF + qrt * kEpiWarpBytes;
    uint32_t hs = 0;
    bool ok = true;
    for (int u = pair; u < n_units && ok; u += n_pairs) {
      const int t0 = u / p.n_mt * unit_rows, w0 = (u % p.n_mt) * 256 + (int)rank * BM + 32 * qrt;
      const int col = w0 + 8 * (lane & 3);
      // the tokens of the unit's rows, 32 in a register across the warp
      int toks[4 * PARTS];
#pragma unroll
      for (int i = 0; i < 4 * PARTS; ++i) {
        const int row = t0 + 32 * i;
        toks[i] = 32 * i < unit_rows && row < rows_used ? __ldg(p.order + row + lane) : p.T;
      }
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        if (h == parts) break;
        const uint32_t b = hs % kSlots;
        ok = __all_sync(kFull, mbar_wait(&accfull[b], (hs / kSlots) & 1, ctl, p.err, p.timeout_ns, 240));
        if (!ok) break;
        tc_fence_after();
        const uint32_t tl = tmem + b * kHalf + ((uint32_t)(qrt * 32) << 16);
#pragma unroll
        for (int j = 0; j < kHalf / 32; ++j) {
          // (a part follows full ones)
          const int jj = 32 * j, tok = toks[h * (kHalf / 32) + j];
          if (jj >= p.n[h]) break;
          if (!__any_sync(kFull, tok < p.T)) continue;
          float v[32];
          tmem_ld32(tl + jj, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t w = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint16_t*>(ebuf + (2 * i) * kEpiPitch + 2 * lane) = (uint16_t)w;
            *reinterpret_cast<uint16_t*>(ebuf + (2 * i + 1) * kEpiPitch + 2 * lane) = (uint16_t)(w >> 16);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2), t = __shfl_sync(kFull, tok, row);
            if (t < p.T && col < p.N)
              *reinterpret_cast<uint4*>(p.out + (size_t)t * p.N + col) =
                  *reinterpret_cast<const uint4*>(ebuf + row * kEpiPitch + 16 * (lane & 3));
          }
          __syncwarp();
        }
        // The issuer needs this warp's TMEM reads only, not its global stores: a relaxed arrival.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0)
            mbar_arrive(&accempty[b]);
          else
            mbar_arrive_cluster_relaxed(accempty_even + 8 * b);
        }
        ++hs;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem, kTmemCols);
  }
}

// =============================================================================
// Input gradient: dx[t] = dY[t] W + q[t] A[a]
// =============================================================================
// The stored rows of W are the reduction here, and its 4-bit codes cannot be
// read along it, so the decoded tile goes to shared memory with the output
// columns contiguous, as the N operand; token rows are the M operand.  Roles per
// CTA: warp 0 codes, warp 1 TMEM owner and (even CTA) UMMA issuer, warp 3
// activation tiles and low-rank operands, warps 4-19 decode groups taking the
// k-chunks round robin, warps 20-23 epilogue; operands of both CTAs are
// counted on the even CTA's barriers, as in the forward.  The low-rank steps
// come after the k-chunks: a unit's two ring slots per adapter (three for 64 ranks)
// hold 64 NB columns of A and both halves of its 128 q rows.
// A unit is 256 rows x 128 NB columns.  NB = 1 where NB = 2 would leave half the
// pairs without one: a unit's chunks are a chain whose step is a decode (training
// step of 777 tokens, 512 -> 2048: 62.7 us with NB = 2, 57.3 us with 1).  8192 rows of
// 2048 columns over 2048: 77 us, 890 TFLOP/s, tensor pipe 50% active: 264 units on 74
// pairs, 42 of them in the fourth turn.
namespace adg {
constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_BYTES = 128 * BK * 2;  // 64 stored rows x 64 NB columns, NB = 2 at most
constexpr int kDecodeWarps = 16;  // in groups of 2 NB, a group's threads a stored row and 64 columns each
constexpr int groups(int nb) { return kDecodeWarps / (2 * nb); }
constexpr int SA = 6;             // activation ring
// Decoded-tile ring: group g's chunks use slot g; codes: two slots a group.  NB = 1 has twice the slots of half the
// bytes.
constexpr int SB = groups(2), RAW_STAGES = 2 * groups(2);
constexpr int RAW_BYTES = 128 * BK / 2;
constexpr int B_OFF = SA * A_BYTES;
constexpr int RAW_OFF = B_OFF + SB * B_BYTES;
constexpr int EPI_OFF = RAW_OFF + RAW_STAGES * RAW_BYTES;
// Epilogue staging, per warp 32 rows x 64 columns; 144-byte rows keep both the row-wise writes and the
// line-wise reads free of bank conflicts.
constexpr int kEpiPitch = 144;
constexpr int kEpiWarpBytes = 32 * kEpiPitch;
constexpr int BAR_OFF = EPI_OFF + 4 * kEpiWarpBytes;
constexpr int SMEM_BYTES = BAR_OFF + 1024 + 1024;
constexpr int kEpiWarp0 = 4 + kDecodeWarps;
constexpr int kThreads = 32 * (kEpiWarp0 + 4);
constexpr int kTmemCols = 512;
static_assert(BAR_OFF % 16 == 0 && SMEM_BYTES <= 232448, "shared memory budget");
static_assert(BM * E4B_MAX_RANK * 2 <= A_BYTES, "low-rank operands fit a slot");
}  // namespace adg

struct AdapterDgradParams {
  const float* absmax;
  const int32_t* order;
  const int32_t* steps;
  uint16_t* out;
  DeviceError* err;
  long long timeout_ns;
  int T, N, K, n, r_pad, n_nt;
};

template <int NB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(adg::kThreads, 1)
    adapter_dgrad_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_raw,
                        const __grid_constant__ CUtensorMap map_la, const __grid_constant__ CUtensorMap map_lb,
                        const AdapterDgradParams p) {
  using namespace adg;
  constexpr int G = groups(NB), RS = 2 * G, kTileSlot = B_BYTES / 2 * NB, kRawSlot = RAW_BYTES / 2 * NB;
  constexpr int kCols = 128 * NB;  // output columns of a unit, 64 NB of them decoded by each CTA
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  uint8_t* aring = smem;
  uint8_t* bring = smem + B_OFF;
  uint8_t* rawbuf = smem + RAW_OFF;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
  uint64_t* raw_full = bars;                    // [RS] codes landed
  uint64_t* raw_empty = raw_full + RS;          // [RS] codes read into registers (group's warps)
  uint64_t* xfull = raw_empty + RS;             // [SA] (even CTA) ring use landed in both CTAs
  uint64_t* aempty = xfull + SA;                // [SA] activation slot consumed by the UMMAs
  uint64_t* bdone = aempty + SA;                // [G] (even CTA) both CTAs' decoded tile written
  uint64_t* bempty = bdone + G;                 // [G] decoded-tile slot consumed by the UMMAs
  uint64_t* accfull = bempty + G;              // [2] accumulator complete
  uint64_t* accempty = accfull + 2;             // [2] (even CTA) accumulator drained in both CTAs
  uint64_t* drain = accfull + 4;                // (even CTA) all issued UMMAs finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accfull + 5);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(accfull + 6);
  uint32_t* sig = reinterpret_cast<uint32_t*>(accfull + 7);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int r = 0; r < RS; ++r) {
      mbar_init(&raw_full[r], 1);
      mbar_init(&raw_empty[r], 2 * NB);
    }
    for (int s = 0; s < SA; ++s) {
      mbar_init(&xfull[s], 1);
      mbar_init(&aempty[s], 1);
    }
    for (int s = 0; s < G; ++s) {
      mbar_init(&bdone[s], 2 * NB);
      mbar_init(&bempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 8);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_2sm(tmem_slot, kTmemCols);
    tmem_relinquish_2sm();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  grid_launch_dependents();

  const int rows_used = p.steps[0];
  const int n_units = (rows_used + kAdapterUnitRows - 1) / kAdapterUnitRows * p.n_nt;
  const int kchunks = (p.N + BK - 1) / BK;
  const int blocks_per_row = p.K / 64;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  const int32_t* granules = p.steps + kAdapterStepsHeader;
  const bool pack = p.r_pad <= 32;  // both halves of the low-rank rows in one slot

  if (warp == 0) {
    // ------------------------------------------------ NF4 codes (one lane)
    if (lane == 0) {
      tma_prefetch_desc(&map_raw);
      uint32_t j = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += n_pairs) {
        const int c0 = (u % p.n_nt) * kCols + (int)rank * 64 * NB;  // this CTA's output columns
        for (int kc = 0; kc < kchunks; ++kc, ++j) {
          const uint32_t r = j % RS, ph = (j / RS) & 1;
          if (!(ok = mbar_wait_lazy(&raw_empty[r], ph ^ 1, ctl, p.err, p.timeout_ns, 311, 64))) break;
          uint8_t* slot = rawbuf + r * kRawSlot;
          mbar_arrive_expect_tx(&raw_full[r], (uint32_t)(2048 * NB));
          tma_load_2d(slot, &map_raw, &raw_full[r], c0 / 2, kc * BK);
          issued |= 1u << r;
          last_par = (last_par & ~(1u << r)) | (ph << r);
        }
      }
      if (!ok) let_land(raw_full, RS, issued, last_par, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------ activation tiles + low-rank operands (one lane)
    if (lane == 0) {
      tma_prefetch_desc(&map_a);
      tma_prefetch_desc(&map_la);
      tma_prefetch_desc(&map_lb);
      const uint32_t xfull_even = mapa_shared(smem_u32(xfull), 0);  // armed there for both CTAs' bytes
      uint32_t s = 0, ph = 0;
      auto issued_next = [&]() {
        if (++s == SA) {
          s = 0;
          ph ^= 1;
        }
      };
      bool ok = true;
      for (int u = pair; u < n_units && ok; u += n_pairs) {
        const int mu = u / p.n_nt, c0 = (u % p.n_nt) * kCols + (int)rank * 64 * NB;
        const int row0 = mu * kAdapterUnitRows + (int)rank * BM;
        AdapterRun<8> run(granules, mu * kAdapterUnitRows, rows_used, kAdapterUnitRows, p.n);
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!(ok = mbar_wait(&aempty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 312))) break;
          if (rank == 0) mbar_arrive_expect_tx(&xfull[s], (uint32_t)(2 * A_BYTES));
          tma_load_2d_pair(aring + s * A_BYTES, &map_a, xfull_even + 8 * s, kc * BK, row0);
          issued_next();
        }
        if (!ok) break;
        while (run.next()) {
          const uint32_t s1 = (s + 1 == SA) ? 0 : s + 1, ph1 = (s + 1 == SA) ? ph ^ 1 : ph;
          const uint32_t s2 = (s1 + 1 == SA) ? 0 : s1 + 1, ph2 = (s1 + 1 == SA) ? ph1 ^ 1 : ph1;
          if (!(ok = mbar_wait(&aempty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 310))) break;
          if (!(ok = mbar_wait(&aempty[s1], ph1 ^ 1, ctl, p.err, p.timeout_ns, 310))) break;
          if (!pack && !(ok = mbar_wait(&aempty[s2], ph2 ^ 1, ctl, p.err, p.timeout_ns, 310))) break;
          uint8_t* lb = aring + s * A_BYTES;
          uint8_t* high = aring + s1 * A_BYTES;
          uint8_t* low = pack ? high + A_BYTES / 2 : aring + s2 * A_BYTES;
          const uint32_t bar = xfull_even + 8 * s;
          if (rank == 0) {
            mbar_arrive_expect_tx(&xfull[s], (uint32_t)((1024 + 256 * NB) * p.r_pad));
            mbar_arrive(&xfull[s1]);
            if (!pack) mbar_arrive(&xfull[s2]);
          }
          tma_load_3d_pair(high, &map_la, bar, 0, 0, row0);
          tma_load_3d_pair(low, &map_la, bar, 0, 1, row0);
          tma_load_3d_pair(lb, &map_lb, bar, c0, 0, run.adapter);
          if (NB == 2) tma_load_3d_pair(lb + 128 * p.r_pad, &map_lb, bar, c0 + 64, 0, run.adapter);
          issued_next();
          issued_next();
          if (!pack) issued_next();
        }
      }
      // (After a wait ran out: copies of either CTA may be in flight; they are given time to land.)
      if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kLandNs) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------ UMMA issuer (even CTA, one elected lane)
    if (elect_one_sync()) {
      const uint32_t idesc = make_idesc_bf16(256, kCols, false, true);
      const uint32_t lswz = swz_for_row_bytes(2 * p.r_pad);
      const uint32_t a_u = smem_u32(aring), b_u = smem_u32(bring);
      const uint32_t bstep = 128u;  // K16 step of the N operand in the descriptor address field
      const uint64_t adesc0 = make_sdesc(a_u, 16, 1024, kSw128);
      const uint64_t bdesc0 = make_sdesc(b_u, 8192, 1024, kSw128);
      uint32_t ti = 0;
      uint32_t sa = 0, pha = 0, sb = 0, phb = 0;
      bool ok = true;
      auto next_a = [&]() {
        if (++sa == SA) {
          sa = 0;
          pha ^= 1;
        }
      };
      auto wait_a = [&]() -> bool { return mbar_wait_cluster(&xfull[sa], pha, ctl, p.err, p.timeout_ns, 323); };
      for (int u = pair; u < n_units && ok; u += n_pairs, ++ti) {
        const int mu = u / p.n_nt;
        AdapterRun<8> run(granules, mu * kAdapterUnitRows, rows_used, kAdapterUnitRows, p.n);
        const uint32_t b = ti & 1, use = ti >> 1;
        const uint32_t d = tmem + b * 256;
        if (!(ok = mbar_wait_cluster(&accempty[b], (use & 1) ^ 1, ctl, p.err, p.timeout_ns, 320))) break;
        tc_fence_after();
        for (int kc = 0; kc < kchunks; ++kc) {
          if (!(ok = wait_a())) break;
          if (!(ok = mbar_wait_cluster(&bdone[sb], phb, ctl, p.err, p.timeout_ns, 324))) break;
          tc_fence_after();
          const uint64_t adesc = adesc0 + (uint64_t)(sa * (A_BYTES >> 4));
          const uint64_t bdesc = bdesc0 + (uint64_t)(sb * (kTileSlot >> 4));
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            umma_bf16_2sm(d, adesc + 2 * kk, bdesc + bstep * kk, idesc, (kc > 0 || kk > 0) ? 1u : 0u);
          umma_commit_2sm(&aempty[sa], 0x3);
          umma_commit_2sm(&bempty[sb], 0x3);
          next_a();
          if (++sb == G) {
            sb = 0;
            phb ^= 1;
          }
        }
        if (!ok) break;
        // One K = r step per adapter of the tile, into its own rows.
        while (run.next()) {
          if (!(ok = wait_a())) break;
          tc_fence_after();
          const uint32_t sa1 = (sa + 1 == SA) ? 0 : sa + 1, sa2 = (sa1 + 1 == SA) ? 0 : sa1 + 1;
          const uint32_t lb_u = a_u + sa * A_BYTES, high = a_u + sa1 * A_BYTES;
          const uint32_t la_u[2] = {high, pack ? high + A_BYTES / 2 : a_u + sa2 * A_BYTES};
          uint32_t off[8];
#pragma unroll
          for (int w = 0; w < 8; ++w) off[w] = rows_off(run.lo, run.hi, w);
          for (int ks = 0; ks < p.r_pad / 16; ++ks) {
            const uint64_t bd = make_sdesc(lb_u + 2048 * ks, 128 * p.r_pad, 1024, kSw128);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              umma_bf16_2sm_masked(d, make_sdesc(la_u[i] + 32 * ks, 16, 16 * p.r_pad, lswz), bd, idesc, off);
          }
          umma_commit_2sm(&aempty[sa], 0x3);
          umma_commit_2sm(&aempty[sa1], 0x3);
          if (!pack) umma_commit_2sm(&aempty[sa2], 0x3);
          next_a();
          next_a();
          if (!pack) next_a();
        }
        if (!ok) break;
        umma_commit_2sm(&accfull[b], 0x3);
      }
      umma_commit_2sm(drain, 0x1);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < kEpiWarp0) {
    // ------------------------------------------------ NF4 decode, groups take the k-chunks round robin
    const uint32_t grp = (warp - 4) / (2 * NB);
    const uint32_t bdone_even = mapa_shared(smem_u32(bdone + grp), 0), sig_even = mapa_shared(smem_u32(sig), 0);
    const int t = (threadIdx.x - 128) & (64 * NB - 1);  // stored row t % 64, block of 64 columns t / 64
    const Nf4Shift ks = nf4_shift_consts();
    const int raw_off = (t & 63) * 32 * NB + (t >> 6) * 32;
    const int drow = t & 63;
    const uint32_t drow_off = (t >> 6) * 8192 + (drow >> 3) * 1024 + (drow & 7) * 128;
    const uint32_t b_u = smem_u32(bring) + grp * kTileSlot;
    // A cursor over this group's chunks, one chunk ahead of the decode (for the block scales).
    const uint32_t my_units = pair < n_units ? (uint32_t)((n_units - pair + n_pairs - 1) / n_pairs) : 0;
    const uint32_t n_chunks = my_units * (uint32_t)kchunks;
    int c_kc = (int)grp, c_u = pair;
    while (c_kc >= kchunks) {
      c_kc -= kchunks;
      c_u += n_pairs;
    }
    int c_nt = c_u % p.n_nt;
    auto advance = [&]() {
      c_kc += G;
      while (c_kc >= kchunks) {
        c_kc -= kchunks;
        c_u += n_pairs;
        c_nt = c_u % p.n_nt;
      }
    };
    // Block scale of this thread's row for the cursor's chunk (0 past the ends of the matrix: zero decode).
    auto block_scale = [&]() -> float {
      if (c_u >= n_units) return 0.0f;
      const int row = c_kc * BK + (t & 63), blk = (c_nt * 2 + (int)rank) * NB + (t >> 6);
      if (row >= p.N || blk >= blocks_per_row) return 0.0f;
      return __ldg(p.absmax + (size_t)row * blocks_per_row + blk);
    };
    float amax_next = block_scale();
    bool ok = true;
    for (uint32_t jj = grp; jj < n_chunks && ok; jj += G) {
      const float amax = amax_next;
      advance();
      const uint32_t r = jj % RS, rph = (jj / RS) & 1;
      ok = __all_sync(kFull, mbar_wait(&raw_full[r], rph, ctl, p.err, p.timeout_ns, 330));
      if (!ok) break;
      const uint8_t* slot = rawbuf + r * kRawSlot;
      const uint4 q0 = *reinterpret_cast<const uint4*>(slot + raw_off);
      const uint4 q1 = *reinterpret_cast<const uint4*>(slot + raw_off + 16);
      const uint32_t codes[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
      fence_proxy_async_smem();  // these reads before the next TMA write of the slot
      __syncwarp();
      if (lane == 0) mbar_arrive(&raw_empty[r]);
      amax_next = block_scale();
      const Nf4Planes pl = nf4_block_planes(amax);
      uint32_t v[32];
#pragma unroll
      for (int c = 0; c < 8; ++c) nf4_decode_word(codes[c], pl, ks, &v[4 * c]);
      ok = __all_sync(kFull, mbar_wait(&bempty[grp], ((jj / G) & 1) ^ 1, ctl, p.err, p.timeout_ns, 331));
      if (!ok) break;
      const uint32_t dbase = b_u + drow_off;
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_shared_v4(dbase + ((c ^ (drow & 7)) << 4), v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      fence_proxy_async_smem();  // the tile stores before the UMMA reads them
      __syncwarp();
      if (lane == 0) {
        if (rank)
          st_async_signal(sig_even, bdone_even, 1u);
        else if (t < 32)
          mbar_arrive_expect_tx(&bdone[grp], 8 * NB);  // and the odd CTA's 2 NB signals of 4 bytes
        else
          mbar_arrive(&bdone[grp]);
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------ epilogue: 32 rows of this warp to their tokens
    // 64 columns at a time through shared memory, so that a store instruction writes whole 128-byte lines
    // of four tokens (a row's columns belong to one lane of TMEM).
    const int qrt = warp & 3;
    const uint32_t accempty_even = mapa_shared(smem_u32(accempty), 0);
    uint8_t* ebuf = smem + EPI_OFF + qrt * kEpiWarpBytes;
    const uint32_t ebuf_u = smem_u32(ebuf) + lane * kEpiPitch;
    uint32_t ti = 0;
    bool ok = true;
    for (int u = pair; u < n_units && ok; u += n_pairs, ++ti) {
      const int mu = u / p.n_nt, c0 = (u % p.n_nt) * kCols;
      const int tok = __ldg(p.order + mu * 256 + (int)rank * 128 + qrt * 32 + lane);
      const uint32_t b = ti & 1, use = ti >> 1;
      ok = __all_sync(kFull, mbar_wait(&accfull[b], use & 1, ctl, p.err, p.timeout_ns, 340));
      if (!ok) break;
      tc_fence_after();
      const bool any = __any_sync(kFull, tok < p.T);
      const uint32_t tl = tmem + b * 256 + ((uint32_t)(qrt * 32) << 16);
#pragma unroll 1
      for (int jj = 0; jj < kCols; jj += 64) {
        if (c0 + jj >= p.K || !any) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[32];
          tmem_ld32(tl + jj + 32 * h, v);
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(ebuf_u + 64 * h + 16 * i, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        __syncwarp();
        const int col = c0 + jj + 8 * (lane & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          const int t = __shfl_sync(kFull, tok, row);
          if (t < p.T && col < p.K)
            *reinterpret_cast<uint4*>(p.out + (size_t)t * p.K + col) =
                *reinterpret_cast<const uint4*>(ebuf + row * kEpiPitch + 16 * (lane & 7));
        }
        __syncwarp();
      }
      // The issuer needs this warp's TMEM reads only, not its global stores: a relaxed arrival.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0)
          mbar_arrive(&accempty[b]);
        else
          mbar_arrive_cluster_relaxed(accempty_even + 8 * b);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_2sm(tmem, kTmemCols);
  }
}

// =============================================================================
// Row gather with the low-rank projection:
//   dst[row] = src[token of row]  (zero for padding rows)
//   out[row] = s[a] dst[row] . F[a], as bf16 pairs (zero for padding rows, whatever the factor holds)
// A task is up to 128 rows of one adapter (or of the tokens without one, which
// are only gathered).  Four loader warps copy the rows' 128-byte pieces into
// the UMMA's swizzled tile with cp.async (zeros for padding rows), the tensor
// core projects the tile, and 16-row bulk stores (a task's rows are a multiple
// of 16, and the next task's rows must not be touched) write it to dst.
// =============================================================================
namespace adp {
constexpr int BM = 128, BK = 64, STAGES = 4;
constexpr int A_BYTES = BM * BK * 2;
constexpr int B_BYTES = BK * E4B_MAX_RANK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 1024;
constexpr int kLoadWarps = 4, kWLoadWarp = 4, kIssueWarp = 5, kStoreWarp = 6, kEpiWarp0 = 7;
constexpr int kThreads = 11 * 32;
constexpr int kAccCols = 64;
constexpr int kTmemCols = 2 * kAccCols;
static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");
static_assert(share_bytes(E4B_MAX_RANK, 8) <= STAGES * STAGE_BYTES, "the shares fit the stages");
static_assert(kAdapterTaskRows == BM, "a task is one tile");
}  // namespace adp

struct AdapterRowsParams {
  const uint16_t* src;   // [T, R]
  const int32_t* order;
  const int32_t* steps;
  const float* scale;
  uint16_t* out;  // [rows, 2, r]
  DeviceError* err;
  long long timeout_ns;
  int R, T, n, r, r_pad, tasks;  // tasks: place of the task list in `steps`
  int S;                         // blocks of a cluster, each a share of R
};

// F = A [n, r, R] (K-major), or B [n, R, r] (W_MN).  With few tasks R is split over the blocks of a cluster: one
// block's chain of chunks would be the launch's time (13 tasks of R = 2048: 21 us, split 8 us).  Reading the rows and
// writing them in their order bounds it: 8192 rows of 2048 columns, 19 us, 3.5 TB/s.
template <bool W_MN>
__global__ void __launch_bounds__(adp::kThreads, 2)
    adapter_proj_kernel(const __grid_constant__ CUtensorMap map_dst, const __grid_constant__ CUtensorMap map_w,
                        const AdapterRowsParams p) {
  using namespace adp;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  uint64_t* full = bars;                  // [STAGES] rows and factor chunk landed
  uint64_t* empty = bars + STAGES;        // [STAGES] read by the UMMAs
  uint64_t* stored = bars + 2 * STAGES;   // [STAGES] read by the bulk stores
  uint64_t* accfull = bars + 3 * STAGES;  // [2]
  uint64_t* accempty = accfull + 2;       // [2]
  uint64_t* drain = accfull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accfull + 5);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(accfull + 6);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], kLoadWarps * 32 + 1);
      mbar_init(&empty[s], 1);
      mbar_init(&stored[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 4);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  grid_launch_dependents();
  const int n_tasks = p.steps[1];
  const int4* tasks = reinterpret_cast<const int4*>(p.steps + p.tasks);  // (adapter, first row, end row, 0)
  const int chunks = (p.R + BK - 1) / BK, rank = (int)blockIdx.x % p.S;
  const int k_lo = rank * chunks / p.S, k_hi = (rank + 1) * chunks / p.S;  // this block's chunks of R
  const int u0 = (int)blockIdx.x / p.S, u_step = (int)gridDim.x / p.S;     // S > 1: one task a cluster
  const uint32_t b_bytes = BK * p.r_pad * 2;
  bool done = false;  // (epilogue warps, S > 1) the accumulator is complete

  if (warp < kLoadWarps) {
    // rows 32 warp + 4 i + lane / 8 of the tile, 16-byte piece lane % 8 of their 128
    const int c = lane & 7;
    uint32_t s = 0, ph = 0;
    bool ok = true;
    for (int u = u0; u < n_tasks && ok; u += u_step) {
      const int4 tk = __ldg(tasks + u);
      const uint16_t* src[8];
      bool live[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = tk.y + 32 * warp + 4 * i + (lane >> 3);
        const int t = row < tk.z ? __ldg(p.order + row) : p.T;
        live[i] = t < p.T;
        src[i] = p.src + (live[i] ? (size_t)t * p.R : 0) + 8 * c;
      }
      for (int kc = k_lo; kc < k_hi; ++kc) {
        if (!(ok = __all_sync(kFull, mbar_wait(&empty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 411)))) break;
        if (!(ok = __all_sync(kFull, mbar_wait(&stored[s], ph ^ 1, ctl, p.err, p.timeout_ns, 412)))) break;
        uint8_t* tile = smem + s * STAGE_BYTES;
        const bool in = kc * BK + 8 * c < p.R;  // the last chunk of a length that is no multiple of 64
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = 32 * warp + 4 * i + (lane >> 3);
          const bool go = live[i] && in;
          cp_async_16_zfill(tile + (q >> 3) * 1024 + (q & 7) * 128 + ((c ^ (q & 7)) << 4),
                            go ? src[i] + kc * BK : p.src, go ? 16u : 0u);
        }
        cp_async_arrive_noinc(&full[s]);
        if (++s == STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight when the shared memory goes away
  } else if (warp == kWLoadWarp) {
    if (lane == 0) {
      tma_prefetch_desc(&map_w);
      uint32_t s = 0, ph = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int u = u0; u < n_tasks && ok; u += u_step) {
        const int a = __ldg(tasks + u).x;
        for (int kc = k_lo; kc < k_hi; ++kc) {
          if (!(ok = mbar_wait(&empty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 413))) break;
          uint8_t* st = smem + s * STAGE_BYTES + A_BYTES;
          if (a < p.n) {
            mbar_arrive_expect_tx(&full[s], b_bytes);
            if (W_MN)
              tma_load_3d(st, &map_w, &full[s], 0, kc * BK, a);
            else
              tma_load_3d(st, &map_w, &full[s], kc * BK, 0, a);
          } else {
            mbar_arrive(&full[s]);  // no adapter: nothing to multiply with
          }
          issued |= 1u << s;
          last_par = (last_par & ~(1u << s)) | (ph << s);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) let_land(full, STAGES, issued, last_par, p.timeout_ns);
    }
  } else if (warp == kIssueWarp) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(BM, p.r_pad, false, W_MN);
      const uint32_t wswz = swz_for_row_bytes(2 * p.r_pad);
      uint32_t s = 0, ph = 0, ti = 0;
      bool ok = true;
      for (int u = u0; u < n_tasks && ok; u += u_step, ++ti) {
        const bool project = __ldg(tasks + u).x < p.n;
        const uint32_t b = ti & 1, use = ti >> 1;
        if (!(ok = mbar_wait(&accempty[b], (use & 1) ^ 1, ctl, p.err, p.timeout_ns, 420))) break;
        tc_fence_after();
        const uint32_t acc = tmem + b * kAccCols;
        for (int kc = k_lo; kc < k_hi; ++kc) {
          if (!(ok = mbar_wait(&full[s], ph, ctl, p.err, p.timeout_ns, 421))) break;
          fence_proxy_async_smem();  // the rows were written by cp.async
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * STAGE_BYTES), b0 = a0 + A_BYTES;
          if (project) {
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
              const uint64_t ad = make_sdesc(a0 + 32 * kk, 16, 1024, kSw128);
              const uint64_t bd = W_MN ? make_sdesc(b0 + 32 * p.r_pad * kk, b_bytes, 16 * p.r_pad, wswz)
                                       : make_sdesc(b0 + 32 * kk, 16, 1024, kSw128);
              umma_bf16(acc, ad, bd, idesc, (kc > k_lo || kk > 0) ? 1u : 0u);
            }
          }
          umma_commit(&empty[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(&accfull[b]);
      }
      umma_commit(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
      }
    }
  } else if (warp == kStoreWarp) {
    // two chunks' stores in flight; a slot is handed back once its stores have read it
    if (lane == 0) {
      tma_prefetch_desc(&map_dst);
      uint32_t s = 0, ph = 0, prev = 0;
      bool ok = true, pending = false;
      for (int u = u0; u < n_tasks && ok; u += u_step) {
        const int4 tk = __ldg(tasks + u);
        const int granules = (min(BM, tk.z - tk.y) + 15) / 16;
        for (int kc = k_lo; kc < k_hi; ++kc) {
          if (!(ok = mbar_wait(&full[s], ph, ctl, p.err, p.timeout_ns, 415))) break;
          fence_proxy_async_smem();
          for (int g = 0; g < granules; ++g)
            tma_store_2d(&map_dst, smem_u32(smem + s * STAGE_BYTES) + g * 2048, kc * BK, tk.y + 16 * g);
          bulk_commit();
          if (pending) {
            bulk_wait_read<1>();
            mbar_arrive(&stored[prev]);
          }
          prev = s;
          pending = true;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      bulk_wait<0>();  // reads and writes of every store done
      if (pending) mbar_arrive(&stored[prev]);
    }
  } else {
    const int q = ((warp & 3) << 5) | lane;  // TMEM lane of this thread
    uint32_t ti = 0;
    bool ok = true;
    for (int u = u0; u < n_tasks && ok; u += u_step, ++ti) {
      const int4 tk = __ldg(tasks + u);
      const bool project = tk.x < p.n;
      const float sc = project ? __ldg(p.scale + tk.x) : 0.0f;
      const uint32_t b = ti & 1, use = ti >> 1;
      const uint32_t tl = tmem + b * kAccCols + ((uint32_t)(32 * (warp & 3)) << 16);
      const int row = tk.y + q;
      const bool live = project && row < tk.z && __ldg(p.order + row) < p.T;
      ok = __all_sync(kFull, mbar_wait(&accfull[b], use & 1, ctl, p.err, p.timeout_ns, 430));
      if (!ok) break;
      tc_fence_after();
      if (p.S > 1) {
        done = project;
        break;
      }
#pragma unroll 1
      for (int j = 0; project && j < p.r_pad; j += 16) {
        float v[16];
        tmem_ld16(tl + j, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = live ? sc * v[i] : 0.0f;
        uint32_t w[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split_bf16x2(v[2 * i], v[2 * i + 1], w[i], l[i]);
        uint16_t* at = p.out + (size_t)row * 2 * p.r + j;
        uint4 *d = reinterpret_cast<uint4*>(at), *e = reinterpret_cast<uint4*>(at + p.r);
        if (row < tk.z) {
          if (j < p.r) {
            d[0] = make_uint4(w[0], w[1], w[2], w[3]);
            e[0] = make_uint4(l[0], l[1], l[2], l[3]);
          }
          if (j + 8 < p.r) {
            d[1] = make_uint4(w[4], w[5], w[6], w[7]);
            e[1] = make_uint4(l[4], l[5], l[6], l[7]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[b]);
    }
  }
  __syncwarp();
  if (p.S > 1) {
    cluster_sync();  // no block's copies or UMMAs use its shared memory any more
    if (done) push_share(smem, tmem, warp & 3, lane, p.S, rank, p.r_pad, true);
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // every share is in place
    const int4 tk = u0 < n_tasks ? __ldg(tasks + u0) : make_int4(p.n, 0, 0, 0);
    const int rows = BM / p.S;
    if (tk.x < p.n && !ctl->abort) {
      const float sc = __ldg(p.scale + tk.x);
      for (int i = threadIdx.x; i < rows * (p.r / 4); i += kThreads) {
        const int row = i % rows, j = 4 * (i / rows), to = tk.y + rank * rows + row;
        if (to < tk.z) {
          uint2 high = make_uint2(0, 0), low = high;
          if (__ldg(p.order + to) < p.T) {
            const float4 v = sum_share(smem, p.S, row, j, p.r_pad);
            split_bf16x2(sc * v.x, sc * v.y, high.x, low.x);
            split_bf16x2(sc * v.z, sc * v.w, high.y, low.y);
          }
          uint16_t* at = p.out + (size_t)to * 2 * p.r + j;
          *reinterpret_cast<uint2*>(at) = high;
          *reinterpret_cast<uint2*>(at + p.r) = low;
        }
      }
    }
  } else {
    __syncthreads();
  }
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// =============================================================================
// Adapter gradients: dA[a] = q^T x (stored transposed), dB[a] = dY^T p
// =============================================================================
// Reading x and dY bounds them.  8192 tokens of 4 adapters of rank 64, 2048 + 2048
// features: 41 us, 1.7 TB/s of their 69 MB: 512 blocks of 8 chunks in two waves, and a
// join of 6 us a cluster.
namespace adw {
constexpr int BM = 128, BK = 64;
constexpr int A_BYTES = BK * BM * 2;  // 64 rows x 128 features, MN-major SW128
// A stage is the features and both halves of 64 rows x r_pad, MN-major; two blocks an SM leave room for four stages
// of up to 32 ranks and three of 64.
constexpr int stages(bool wide) { return wide ? 3 : 4; }
constexpr int half_bytes(bool wide) { return BK * (wide ? E4B_MAX_RANK : E4B_MAX_RANK / 2) * 2; }
constexpr int stage_bytes(bool wide) { return A_BYTES + 2 * half_bytes(wide); }
constexpr int smem_bytes(bool wide) { return stages(wide) * stage_bytes(wide) + 1024 + 1024; }
// warps 0-3 row loaders, 4 low-rank rows, 5 UMMA issuer + TMEM owner, 6-9 epilogue
constexpr int kLoadWarps = 4, kLowWarp = 4, kIssueWarp = 5;
constexpr int kThreads = 10 * 32;
constexpr int kAccCols = 64;
constexpr int kTmemCols = 2 * kAccCols;
static_assert(stage_bytes(false) % 1024 == 0 && stage_bytes(true) % 1024 == 0, "stage alignment");
static_assert(share_bytes(E4B_MAX_RANK, 8) <= stages(true) * stage_bytes(true) &&
                  share_bytes(E4B_MAX_RANK / 2, 8) <= stages(false) * stage_bytes(false),
              "the shares fit the stages");
}  // namespace adw

struct AdapterWgradParams {
  const uint16_t* act[2];  // x [T, K], dY [T, N]
  uint16_t* out[2];  // dA [n, r, K], dB [n, N, r]
  int F[2], n_ft[2];
  const int32_t* order;
  const int32_t* offsets;
  DeviceError* err;
  long long timeout_ns;
  int T, n, r, r_pad;
  int S;  // blocks of a cluster, each a share of an adapter's rows
};

struct AdapterWgradUnit {
  int g, ft, a, row0, rows;  // rows: all of the adapter's
  int k_lo, k_hi;            // this block's 64-row chunks of them
};
__device__ __forceinline__ AdapterWgradUnit adapter_wgrad_unit(const AdapterWgradParams& p, int u) {
  AdapterWgradUnit w;
  const int per = p.n_ft[0] + p.n_ft[1];
  w.a = u / per;
  w.ft = u - w.a * per;
  w.g = w.ft >= p.n_ft[0];
  if (w.g) w.ft -= p.n_ft[0];
  w.row0 = __ldg(p.offsets + w.a);
  w.rows = __ldg(p.offsets + w.a + 1) - w.row0;  // a multiple of 32
  const int chunks = (w.rows + adw::BK - 1) / adw::BK, rank = (int)blockIdx.x % p.S;
  w.k_lo = rank * chunks / p.S;
  w.k_hi = (rank + 1) * chunks / p.S;
  return w;
}

template <bool WIDE>  // r > 32
__global__ void __launch_bounds__(adw::kThreads, 2)
    adapter_wgrad_kernel(const __grid_constant__ CUtensorMap low0, const __grid_constant__ CUtensorMap low1,
                         const AdapterWgradParams p) {
  using namespace adw;
  constexpr int STAGES = stages(WIDE), HALF_BYTES = half_bytes(WIDE), STAGE_BYTES = stage_bytes(WIDE);
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = align1024(smem_dyn);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  uint64_t* full = bars;
  uint64_t* empty = bars + STAGES;
  uint64_t* accfull = bars + 2 * STAGES;  // [2]
  uint64_t* accempty = accfull + 2;       // [2]
  uint64_t* drain = accfull + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accfull + 5);
  CtaControl* ctl = reinterpret_cast<CtaControl*>(accfull + 6);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], kLoadWarps * 32 + 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accfull[b], 1);
      mbar_init(&accempty[b], 4);
    }
    mbar_init(drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();
  grid_launch_dependents();
  const int n_units = p.n * (p.n_ft[0] + p.n_ft[1]);
  const uint32_t b_bytes = BK * p.r_pad * 2;
  const int u0 = (int)blockIdx.x / p.S, u_step = (int)gridDim.x / p.S;  // S > 1: one unit a cluster
  bool done = false;  // (epilogue warps, S > 1) the accumulator is complete

  if (warp < kLoadWarps) {
    // rows 16 warp + 4 (i % 4) + lane / 8 of the chunk, feature half i / 4, 16-byte piece lane % 8
    const int c = lane & 7;
    uint32_t s = 0, ph = 0;
    bool ok = true;
    for (int u = u0; u < n_units && ok; u += u_step) {
      const AdapterWgradUnit w = adapter_wgrad_unit(p, u);
      const uint16_t* act = w.g ? p.act[1] : p.act[0];
      const int F = w.g ? p.F[1] : p.F[0];
      const int f = w.ft * BM + 8 * c;
      auto tokens = [&](int kc, int (&t)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = kc * BK + 16 * warp + 4 * i + (lane >> 3);
          t[i] = row < w.rows ? __ldg(p.order + w.row0 + row) : p.T;
        }
      };
      int t[4], t1[4];  // of this chunk and the next: their loads have a chunk's time
      tokens(w.k_lo, t);
      tokens(w.k_lo + 1, t1);
      for (int kc = w.k_lo; kc < w.k_hi; ++kc) {
        if (!(ok = __all_sync(kFull, mbar_wait(&empty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 510)))) break;
        uint8_t* tile = smem + s * STAGE_BYTES;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int q = 16 * warp + 4 * (i & 3) + (lane >> 3), col = f + 64 * (i >> 2);
          const bool go = t[i & 3] < p.T && col < F;
          cp_async_16_zfill(tile + (i >> 2) * (A_BYTES / 2) + (q >> 3) * 1024 + (q & 7) * 128 + ((c ^ (q & 7)) << 4),
                            go ? act + (size_t)t[i & 3] * F + col : act, go ? 16u : 0u);
        }
        cp_async_arrive_noinc(&full[s]);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = t1[i];
        tokens(kc + 2, t1);
        if (++s == STAGES) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == kLowWarp) {
    if (lane == 0) {
      uint32_t s = 0, ph = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += u_step) {
        const AdapterWgradUnit w = adapter_wgrad_unit(p, u);
        const CUtensorMap* low = w.g ? &low1 : &low0;
        for (int kc = w.k_lo; kc < w.k_hi; ++kc) {
          if (!(ok = mbar_wait(&empty[s], ph ^ 1, ctl, p.err, p.timeout_ns, 511))) break;
          mbar_arrive_expect_tx(&full[s], 2 * b_bytes);
          uint8_t* b = smem + s * STAGE_BYTES + A_BYTES;
          tma_load_3d(b, low, &full[s], 0, 0, w.row0 + kc * BK);
          tma_load_3d(b + HALF_BYTES, low, &full[s], 0, 1, w.row0 + kc * BK);
          issued |= 1u << s;
          last_par = (last_par & ~(1u << s)) | (ph << s);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) let_land(full, STAGES, issued, last_par, p.timeout_ns);
    }
  } else if (warp == kIssueWarp) {
    if (lane == 0) {
      const uint32_t idesc = make_idesc_bf16(BM, p.r_pad, true, true);
      const uint32_t lswz = swz_for_row_bytes(2 * p.r_pad);
      int s = 0;
      uint32_t ph = 0, ti = 0;
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += u_step, ++ti) {
        const AdapterWgradUnit w = adapter_wgrad_unit(p, u);
        const uint32_t b = ti & 1, use = ti >> 1;
        if (!(ok = mbar_wait(&accempty[b], (use & 1) ^ 1, ctl, p.err, p.timeout_ns, 520))) break;
        tc_fence_after();
        const uint32_t acc = tmem + b * kAccCols;
        for (int kc = w.k_lo; kc < w.k_hi; ++kc) {
          if (!(ok = mbar_wait(&full[s], ph, ctl, p.err, p.timeout_ns, 521))) break;
          fence_proxy_async_smem();  // the rows were written by cp.async
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * STAGE_BYTES), b0 = a0 + A_BYTES;
          const int steps = min(BK, w.rows - kc * BK) / 16;  // rows past the adapter's end take no part
          for (int kk = 0; kk < steps; ++kk) {
            const uint64_t ad = make_sdesc(a0 + 2048 * kk, A_BYTES / 2, 1024, kSw128);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint64_t bd = make_sdesc(b0 + i * HALF_BYTES + 32 * p.r_pad * kk, b_bytes, 16 * p.r_pad, lswz);
              umma_bf16(acc, ad, bd, idesc, (kc > w.k_lo || kk > 0 || i > 0) ? 1u : 0u);
            }
          }
          umma_commit(&empty[s]);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(&accfull[b]);
      }
      umma_commit(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && (long long)(globaltimer_ns() - t0) < p.timeout_ns) {
      }
    }
  } else {
    const int q = ((warp & 3) << 5) | lane;
    uint32_t ti = 0;
    bool ok = true;
    for (int u = u0; u < n_units && ok; u += u_step, ++ti) {
      const AdapterWgradUnit w = adapter_wgrad_unit(p, u);
      const uint32_t b = ti & 1, use = ti >> 1;
      const uint32_t tl = tmem + b * kAccCols + ((uint32_t)(32 * (warp & 3)) << 16);
      ok = __all_sync(kFull, mbar_wait(&accfull[b], use & 1, ctl, p.err, p.timeout_ns, 530));
      if (!ok) break;
      tc_fence_after();
      if (p.S > 1) {
        done = true;
        break;
      }
      const int F = p.F[w.g], m = w.ft * BM + q;
      uint16_t* out = p.out[w.g];
#pragma unroll 1
      for (int j = 0; j < p.r_pad; j += 16) {
        float v[16];
        if (w.rows > 0) {
          tmem_ld16(tl + j, v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        }
        if (m < F) {
          if (w.g) {  // dB [N, r]
            uint32_t pw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) pw[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            uint4* d = reinterpret_cast<uint4*>(out + ((size_t)w.a * F + m) * p.r + j);
            if (j < p.r) d[0] = make_uint4(pw[0], pw[1], pw[2], pw[3]);
            if (j + 8 < p.r) d[1] = make_uint4(pw[4], pw[5], pw[6], pw[7]);
          } else {  // dA [r, K]: lanes write neighbouring features
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (j + i < p.r) {
                const __nv_bfloat16 h = __float2bfloat16_rn(v[i]);
                out[((size_t)w.a * p.r + j + i) * F + m] = *reinterpret_cast<const uint16_t*>(&h);
              }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[b]);
    }
  }
  __syncwarp();
  if (p.S > 1) {
    const AdapterWgradUnit w = adapter_wgrad_unit(p, u0);  // the grid holds n_units clusters
    const int rank = (int)blockIdx.x % p.S, rows = BM / p.S, F = w.g ? p.F[1] : p.F[0];
    cluster_sync();  // no block's copies or UMMAs use its shared memory any more
    if (done) push_share(smem, tmem, warp & 3, lane, p.S, rank, p.r_pad, w.k_hi > w.k_lo);
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // every share is in place
    if (!ctl->abort) {
      const int m0 = w.ft * BM + rank * rows;
      uint16_t* out = w.g ? p.out[1] : p.out[0];
      for (int i = threadIdx.x; i < rows * (p.r / 4); i += kThreads) {
        const int row = i % rows, j = 4 * (i / rows), m = m0 + row;  // neighbouring threads: neighbouring features
        if (m >= F) continue;
        const float4 v = sum_share(smem, p.S, row, j, p.r_pad);
        const uint32_t lo = pack_bf16x2(v.x, v.y), hi = pack_bf16x2(v.z, v.w);
        if (w.g) {
          *reinterpret_cast<uint2*>(out + ((size_t)w.a * F + m) * p.r + j) = make_uint2(lo, hi);
        } else {
          uint16_t* d = out + ((size_t)w.a * p.r + j) * F + m;
          d[0] = (uint16_t)lo;
          d[F] = (uint16_t)(lo >> 16);
          d[2 * (size_t)F] = (uint16_t)hi;
          d[3 * (size_t)F] = (uint16_t)(hi >> 16);
        }
      }
    }
  } else {
    __syncthreads();
  }
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// =============================================================================
// Host-side launchers
// =============================================================================
namespace {
int rank_padded(int r) { return r <= 16 ? 16 : (r <= 32 ? 32 : 64); }

// launch_following with the kernel's limit of dynamic shared memory set to `smem`, the same in every call.
template <typename... Params, typename... Args>
cudaError_t launch_tiles(void (*kernel)(Params...), int grid, int threads, int smem, int S, cudaStream_t stream,
                         const Args&... args) {
  const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  return err != cudaSuccess ? err : launch_following(kernel, grid, threads, smem, S, stream, args...);
}

// 2-D byte matrix [rows, bytes].
cudaError_t map_u8_2d(CUtensorMap* m, const void* base, uint64_t bytes, uint64_t rows, uint32_t box_bytes,
                      uint32_t box_rows) {
  const uint64_t dims[2] = {bytes, rows};
  const uint64_t strides[1] = {bytes};
  const uint32_t box[2] = {box_bytes, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_NONE);
}
// Halves of p or q, bf16 [rows, 2, r]: a tile is one half of `box_rows` rows.
cudaError_t map_halves(CUtensorMap* m, const void* base, int r, uint64_t rows, int r_pad, uint32_t box_rows) {
  const uint64_t dims[3] = {(uint64_t)r, 2, rows};
  const uint64_t strides[2] = {(uint64_t)r * 2, (uint64_t)r * 4};
  const uint32_t box[3] = {(uint32_t)r_pad, 1, box_rows};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                           swizzle_for_bytes(2 * r_pad));
}
}  // namespace

// Token rows of a forward unit: the ones that take the pairs the least time.  Measured cycles a 64-wide chunk: 680 up
// to 128 rows (decoding it), 790 with 160, 840 with 256, 1400 with 384.
static int fwd_unit_rows(const AdapterProjHost& h, int n_mt, int pairs) {
  const int64_t rows = h.T + 16 * (int64_t)(h.T < h.n + 1 ? h.T : h.n + 1);  // with an average of padding
  int best = 256;
  int64_t best_cost = INT64_MAX;
  for (int nt = 384; nt >= 96; nt -= 32) {
    const int64_t turns = ((rows + nt - 1) / nt * n_mt + pairs - 1) / pairs;
    if (nt > 256 && turns > 1) continue;  // all three accumulator slots: nothing left for a next unit
    const int64_t cost = turns * (nt > 256 ? 1400 : nt > 128 ? 707 + 13 * nt / 25 : 680);
    if (cost < best_cost) {
      best = nt;
      best_cost = cost;
    }
  }
  return best;
}

cudaError_t launch_adapter_fwd(const AdapterProjHost& h, const uint16_t* rows, const uint16_t* low, const uint16_t* B,
                               uint16_t* y, int num_sms, cudaStream_t stream) {
  const int rp = rank_padded(h.r);
  const CUtensorMapSwizzle rswz = swizzle_for_bytes(2 * rp);
  const int n_mt = (h.N + 255) / 256, unit_rows = fwd_unit_rows(h, n_mt, num_sms / 2);
  AdapterFwdParams p;
  int last = 0;
  for (int i = 0; i < 3; ++i) {
    const int left = unit_rows - i * adf::kHalf;
    p.n[i] = left <= 0 ? 0 : (left < adf::kHalf ? left : adf::kHalf);
    if (p.n[i]) last = p.n[i];
  }
  CUtensorMap mx0, mx1, mraw, mp, mb;
  cudaError_t err;
  if ((err = map_bf16_2d(&mx0, rows, h.K, h.rows_cap, 64, p.n[0] / 2, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
    return err;
  if ((err = map_bf16_2d(&mx1, rows, h.K, h.rows_cap, 64, last / 2, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess)
    return err;
  if ((err = map_u8_2d(&mraw, h.nf4, h.K / 2, h.N, 32, 128)) != cudaSuccess) return err;
  if ((err = map_halves(&mp, low, h.r, h.rows_cap, rp, 16)) != cudaSuccess) return err;
  if ((err = map_bf16_3d(&mb, B, h.r, h.N, h.n, rp, 64, rswz)) != cudaSuccess) return err;
  p.absmax = h.absmax;
  p.order = h.order;
  p.steps = h.steps;
  p.out = y;
  p.err = h.err;
  p.timeout_ns = h.timeout_ns;
  p.K = h.K;
  p.N = h.N;
  p.T = h.T;
  p.r_pad = rp;
  p.n_adapters = h.n;
  p.n_mt = n_mt;
  const int64_t units = (h.rows_cap + unit_rows - 1) / unit_rows * n_mt;
  const int grid = 2 * (int)(units < num_sms / 2 ? units : num_sms / 2);
  LaunchScope scope("adapter_fwd", stream);
  return launch_tiles(p.n[2] ? adapter_fwd_kernel<3> : adapter_fwd_kernel<2>, grid, adf::threads(p.n[2] ? 3 : 2),
                      adf::SMEM_BYTES, 0, stream, mx0, mx1, mraw, mp, mb, p);
}

cudaError_t launch_adapter_dgrad(const AdapterProjHost& h, const uint16_t* rows, const uint16_t* low,
                                 const uint16_t* A, uint16_t* dx, int num_sms, cudaStream_t stream) {
  const int rp = rank_padded(h.r);
  CUtensorMap ma, mraw, mla, mlb;
  cudaError_t err;
  if ((err = map_bf16_2d(&ma, rows, h.N, h.rows_cap, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return err;
  const int64_t row_units = h.rows_cap / kAdapterUnitRows;
  const int nb = 2 * row_units * ((h.K + 255) / 256) <= num_sms / 2 ? 1 : 2;
  if ((err = map_u8_2d(&mraw, h.nf4, h.K / 2, h.N, 32 * nb, 64)) != cudaSuccess) return err;
  if ((err = map_halves(&mla, low, h.r, h.rows_cap, rp, 128)) != cudaSuccess) return err;
  if ((err = map_bf16_3d(&mlb, A, h.K, h.r, h.n, 64, rp, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return err;
  AdapterDgradParams p;
  p.absmax = h.absmax;
  p.order = h.order;
  p.steps = h.steps;
  p.out = dx;
  p.err = h.err;
  p.timeout_ns = h.timeout_ns;
  p.T = h.T;
  p.N = h.N;
  p.K = h.K;
  p.r_pad = rp;
  p.n = h.n;
  p.n_nt = (h.K + 128 * nb - 1) / (128 * nb);
  const int64_t units = row_units * p.n_nt;
  const int grid = 2 * (int)(units < num_sms / 2 ? units : num_sms / 2);
  LaunchScope scope("adapter_dgrad", stream);
  return launch_tiles(nb == 1 ? adapter_dgrad_kernel<1> : adapter_dgrad_kernel<2>, grid, adg::kThreads,
                          adg::SMEM_BYTES, 0, stream, ma, mraw, mla, mlb, p);
}

cudaError_t launch_adapter_rows(const AdapterProjHost& h, bool mn, const uint16_t* src, const uint16_t* fac,
                                uint16_t* rows, uint16_t* out, int num_sms, cudaStream_t stream) {
  const int R = mn ? h.N : h.K, rp = rank_padded(h.r);
  CUtensorMap ms, mw;
  cudaError_t err;
  if ((err = map_bf16_2d(&ms, rows, R, h.rows_cap, 64, 16, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return err;
  if (mn)  // B [n, N, r]
    err = map_bf16_3d(&mw, fac, h.r, h.N, h.n, rp, 64, swizzle_for_bytes(2 * rp));
  else  // A [n, r, K]
    err = map_bf16_3d(&mw, fac, h.K, h.r, h.n, 64, rp, CU_TENSOR_MAP_SWIZZLE_128B);
  if (err != cudaSuccess) return err;
  AdapterRowsParams p;
  p.src = src;
  p.n = h.n;
  p.order = h.order;
  p.steps = h.steps;
  p.scale = h.scale;
  p.out = out;
  p.err = h.err;
  p.timeout_ns = h.timeout_ns;
  p.R = R;
  p.T = h.T;
  p.r = h.r;
  p.r_pad = rp;
  p.tasks = (int)adapter_tasks_offset(h.rows_cap);
  // two blocks an SM; R is split while all clusters fit at once and every block keeps two chunks
  const int64_t cap = h.rows_cap / kAdapterTaskRows + h.n + 1, fit = 2 * (int64_t)num_sms;
  const int chunks = (R + adp::BK - 1) / adp::BK;
  p.S = 1;
  while (p.S < 8 && 2 * p.S * cap <= fit && chunks >= 4 * p.S) p.S *= 2;
  const int grid = p.S * (int)(cap < fit / p.S ? cap : fit / p.S);
  LaunchScope scope(mn ? "adapter_proj_dy" : "adapter_proj_x", stream);
  return mn ? launch_tiles(adapter_proj_kernel<true>, grid, adp::kThreads, adp::SMEM_BYTES, p.S, stream, ms, mw, p)
            : launch_tiles(adapter_proj_kernel<false>, grid, adp::kThreads, adp::SMEM_BYTES, p.S, stream, ms, mw,
                              p);
}

cudaError_t launch_adapter_wgrad(const AdapterProjHost& h, const uint16_t* x, const uint16_t* dY, const uint16_t* p_low,
                                 const uint16_t* q_low, uint16_t* dA, uint16_t* dB, int num_sms, cudaStream_t stream) {
  const int rp = rank_padded(h.r);
  CUtensorMap mq, mp;
  cudaError_t err;
  if ((err = map_halves(&mq, q_low, h.r, h.rows_cap, rp, 64)) != cudaSuccess) return err;
  if ((err = map_halves(&mp, p_low, h.r, h.rows_cap, rp, 64)) != cudaSuccess) return err;
  AdapterWgradParams p;
  p.act[0] = x;
  p.act[1] = dY;
  p.out[0] = dA;
  p.out[1] = dB;
  p.F[0] = h.K;
  p.F[1] = h.N;
  p.n_ft[0] = (h.K + adw::BM - 1) / adw::BM;
  p.n_ft[1] = (h.N + adw::BM - 1) / adw::BM;
  p.order = h.order;
  p.offsets = h.offsets;
  p.err = h.err;
  p.timeout_ns = h.timeout_ns;
  p.T = h.T;
  p.n = h.n;
  p.r = h.r;
  p.r_pad = rp;
  // Rows are split over clusters where that fills the GPU twice over (adapters have unequal numbers of rows) and
  // leaves a block four chunks of an even share.
  const int64_t units = (int64_t)h.n * (p.n_ft[0] + p.n_ft[1]), cap = (int64_t)num_sms * 2;
  p.S = 1;
  while (p.S < 8 && 2 * p.S * units <= 2 * cap && h.T / h.n >= 8 * p.S * adw::BK) p.S *= 2;
  const int grid = (int)(p.S > 1 ? units * p.S : (units < cap ? units : cap));
  LaunchScope scope("adapter_wgrad", stream);
  return rp > 32 ? launch_tiles(adapter_wgrad_kernel<true>, grid, adw::kThreads, adw::smem_bytes(true), p.S, stream,
                                mq, mp, p)
                 : launch_tiles(adapter_wgrad_kernel<false>, grid, adw::kThreads, adw::smem_bytes(false), p.S, stream,
                                mq, mp, p);
}

}  // namespace e4b
