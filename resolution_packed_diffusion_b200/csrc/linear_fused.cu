// linear_fused.cu -- the modality-specific linear layer with its epilogue in the
// product's kernel, and its backward, on sm_100a tensor cores:
//   z[t] = x[t] W[m]^T + b[m],  out[t] = act(z[t]) + resid[t]
//   dz = dout * act'(z),  dx[t] = dz[t] W[m],  dW[m] = sum_t dz[t]^T x[t],  db[m] = sum_t dz[t]
// with m the token's modality (0 image, 1 text), W stored [2][N][K], sums over
// the modality's tokens. z may be kept for the backward in bf16 or as an 8-bit
// checkpoint (act8.cu), written by the same epilogue; the backward takes x and z
// in either form.
// Source (page title, section): picx.dev "Mage-Flow" summary, Methodology >
// Native-Resolution MMDiT (each stream keeps its own weights) and > Training
// Infrastructure (the packed model is trained).
//
// One kernel template carries the three products (clusters of two CTAs on two
// SMs, cta_group::2: 256 x 256 output tiles as M = 256, N = 256 MMAs with fp32
// accumulators in TMEM, 64 of the inner dimension per stage); the backward's two run
// in one launch, their tiles in one queue, the longest first, so that neither leaves
// SMs idle at its end. Nothing is transposed in memory: the operands are read as they
// lie, and the tensor core's descriptors say which way they run.
//   forward  A = x (inner dimension contiguous), B = W (contiguous)
//   dx       A = dz (contiguous),                B = W (inner dimension strided)
//   dW       A = dz, B = x (both strided: the inner dimension is the tokens)
// W has a three-dimensional tensor map (K, N, modality), so a tile past N or K
// reads zeros and not the other modality's weights. Tails need no padding: rows
// and columns past the end are read as zeros and not stored.
//
// The sum over a modality's tokens walks its runs of consecutive rows (an image,
// a text) in steps of 64. The last step of a run may reach into rows of the other
// modality; there the rows past the run are set to zero in shared memory, in both
// operands, between the copies and the MMAs, so that an infinity or NaN in a
// foreign row has no effect. Whole steps go from the copies to the MMAs directly:
// sending every step through a warp that hands it on across the pair cost 1.0 us a
// step against 0.39 (the whole of dW 1253 us against 494).
//   warp 0      TMA producer (all lanes in the loop, one issues)
//   warp 1      tcgen05 issuer (likewise, in the leader CTA)
//   warp 2      backward: zeroes the rows past a run
//   warp 3      backward: adds the partial sums of db that dz_kernel left
//   warps 4..11 epilogue, from the accumulator that the MMAs have left for the other
//               one of the two: one output row and half of the columns per thread
// Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "act8.cuh"
#include "gemm_internal.h"
#include "linear_common.cuh"
#include "mf_internal.h"
#include "mf_ptx.cuh"
#include "mlp_internal.h"
#include "pdl.cuh"

namespace mf {

namespace {

constexpr int kFwd = 0, kBwd = 1;
constexpr int kHalf = 128;   // output rows, and B columns, of one CTA of the pair
constexpr int kTile = 256;   // output tile: rows, and columns at most
constexpr int kStepK = 64;   // inner dimension per stage: one 128-byte swizzle atom
constexpr int kBoxBytes = 64 * 64 * 2;  // a 64-column box of 64 rows
constexpr uint32_t kTmemCols = 512;     // two accumulators of 256 columns
constexpr int kWarps = 12;

constexpr int kStages = 7;
constexpr int kABytes = kHalf * kStepK * 2;
constexpr int kStageBytes = 2 * kABytes;  // A and B, as copied into one CTA

// Barriers. FULL (the leader's) counts both CTAs' producers and the bytes of both
// CTAs' copies; for a step that needs rows zeroed the copies complete on their own
// CTA's PART, and the zeroing warps arrive on FULL in the producers' place. EMPTY
// and ACC_FULL arrive in both CTAs from the leader's multicast commits; ACC_EMPTY,
// the leader's, counts both CTAs' epilogue warps.
constexpr int kFull = 0;
constexpr int kEmpty = kFull + kStages;
constexpr int kPart = kEmpty + kStages;
constexpr int kAccFull = kPart + kStages;
constexpr int kAccEmpty = kAccFull + 2;
constexpr int kDrain = kAccEmpty + 2;
constexpr int kNumBars = kDrain + 1;
constexpr int kOffBar = kStages * kStageBytes;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // TMEM address, abort flag
constexpr int kOffBias = kOffMisc + 16;           // the tile's bias: 256 floats
constexpr int kSmemBytes = kOffBias + kTile * 4 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory budget of one CTA");

// out[c] = the sum of part[k][c] over k, in order.
struct ColumnSums {
  const float* part;
  int32_t n, cols;
  float* out;
};

// The column tiles of a product's output.
struct Columns {
  int32_t width;  // columns of a tile: a multiple of 16, at most 256
  int32_t tiles;
  int32_t nb;     // tiles per block of the traversal
};

struct FwdArgs {
  GemmJobs jobs;   // one per (row block, modality present in it)
  int32_t T, K, N;
  Columns cols;
  const uint8_t* tok_mod;
  LinearEpilogue ep;
  KernelCtl ctl;
};

// Kinds of the backward's units.
constexpr int kDx = 0, kDwImage = 1;  // kDwImage + 1: dW of the text modality

struct BwdArgs {
  GemmJobs jobs;  // dx
  // dW: the modalities' runs; it0[m][r] = steps before run r
  int32_t n[2];
  int32_t start[2][MF_MAX_SAMPLES];
  int32_t len[2][MF_MAX_SAMPLES];
  int32_t it0[2][MF_MAX_SAMPLES + 1];
  int32_t splits[2];    // parts of the modality's steps
  int32_t slot0[2];     // the modality's first slot of partial sums
  float* part;          // [slots][256][256]
  int32_t kind[3];      // the kinds in the queue's order, and where each ends in it
  int32_t end[3];
  int32_t T, K, N;
  Columns dx_cols, dw_cols;
  const uint8_t* tok_mod;
  mf_bf16* dx;
  mf_bf16* dW;
  ColumnSums db;        // db's partials, or out NULL
  KernelCtl ctl;
};

template <int MODE>
struct ArgsOf {
  using type = FwdArgs;
};
template <>
struct ArgsOf<kBwd> {
  using type = BwdArgs;
};

// Unit u -> (row tile or job, column tile): blocks of nb column tiles (the last
// one may be narrower), inside a block every row in turn. The units in flight
// share a block's B operand in L2 while A streams past it.
__device__ __forceinline__ void unit_coords(int u, int rows, int cols, int nb, int& r, int& c) {
  const int per = rows * nb;
  const int b = u / per;
  const int w = min(nb, cols - b * nb);
  const int i = u - b * per;
  r = i / w;
  c = b * nb + (i - r * w);
}

// Arrives on a barrier of either CTA of the pair and adds `bytes` to what it
// expects.
__device__ __forceinline__ void expect_pair(bool leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// A box of the weights: modality z of the (K, N, 2) map, completing on the
// leader's barrier; kept in L2 (evict_last) since every row block reads it.
__device__ __forceinline__ void load_w(bool leader, void* dst, const CUtensorMap* map,
                                       uint32_t bar, int x, int y, int z, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const KernelCtl& ctl,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, abort_flag));
}

// mbar_wait for arrivals of both CTAs that release writes to their shared memory:
// acquires at cluster scope. (A cluster fence after a plain wait does the same and
// costs the issuing thread about a microsecond a step.)
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  const KernelCtl& ctl, volatile int* abort_flag) {
  if (try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > ctl.wait_limit_ns) {
      *abort_flag = 1;
      atomicCAS(ctl.err, 0, static_cast<int>(MF_ERR_TIMEOUT));
      return false;
    }
  }
}

// What a unit covers. Forward and dx: row block, modality, column tile, all steps of
// the inner dimension. dW: modality, row tile (blk), column tile, steps [s0, s0 +
// steps) of the modality's runs (none without tokens), slot of its partial sums (-1:
// dW itself).
struct Unit {
  bool dw;
  int blk, m, ct, s0, steps, slot;
};
__device__ __forceinline__ Unit unit_of(const FwdArgs& a, int u) {
  Unit w;
  int ji;
  unit_coords(u, a.jobs.n, a.cols.tiles, a.cols.nb, ji, w.ct);
  const int job = a.jobs.job[ji];
  w.dw = false;
  w.blk = job & 0x7fff;
  w.m = job >> 15;
  w.s0 = 0;
  w.steps = (a.K + kStepK - 1) / kStepK;
  w.slot = -1;
  return w;
}
__device__ __forceinline__ Unit unit_of(const BwdArgs& a, int u) {
  Unit w;
  const int q = (u >= a.end[0]) + (u >= a.end[1]);
  const int kind = a.kind[q];
  if (q > 0) u -= a.end[q - 1];
  if (kind == kDx) {
    int ji;
    unit_coords(u, a.jobs.n, a.dx_cols.tiles, a.dx_cols.nb, ji, w.ct);
    const int job = a.jobs.job[ji];
    w.dw = false;
    w.blk = job & 0x7fff;
    w.m = job >> 15;
    w.s0 = 0;
    w.steps = (a.N + kStepK - 1) / kStepK;
    w.slot = -1;
    return w;
  }
  w.dw = true;
  w.m = kind - kDwImage;
  const int rows = (a.N + kTile - 1) / kTile;
  const int tiles = rows * a.dw_cols.tiles;
  const int part = u / tiles;
  unit_coords(u - part * tiles, rows, a.dw_cols.tiles, a.dw_cols.nb, w.blk, w.ct);
  const int total = a.it0[w.m][a.n[w.m]], p = a.splits[w.m];
  w.s0 = static_cast<int>(static_cast<int64_t>(total) * part / p);
  w.steps = static_cast<int>(static_cast<int64_t>(total) * (part + 1) / p) - w.s0;
  w.slot = p > 1 ? a.slot0[w.m] + part * tiles + w.blk * a.dw_cols.tiles + w.ct : -1;
  return w;
}
// The walk over a dW unit's steps: run and first row of the current one.
struct RunWalk {
  int r, row, left;
  template <class A>
  __device__ __forceinline__ void start(const A& a, const Unit& w) {
    int lo = 0, hi = a.n[w.m] - 1;  // last run with it0 <= s0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.it0[w.m][mid] <= w.s0) lo = mid; else hi = mid - 1;
    }
    r = lo;
    const int off = (w.s0 - a.it0[w.m][r]) * kStepK;
    row = a.start[w.m][r] + off;
    left = a.len[w.m][r] - off;
  }
  template <class A>
  __device__ __forceinline__ void next(const A& a, int m) {
    row += kStepK;
    left -= kStepK;
    if (left <= 0 && r + 1 < a.n[m]) {
      ++r;
      row = a.start[m][r];
      left = a.len[m][r];
    }
  }
};

template <int ACT>
__device__ __forceinline__ void act32(float (&v)[32]) {
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const uint64_t r = act_fwd2<ACT>(f2_pack(v[e], v[e + 1]));
    f2_unpack(r, v[e], v[e + 1]);
  }
}

// 32 columns' bias, the same for every row: broadcast reads of shared memory.
__device__ __forceinline__ void add_bias32(const float* bias, float (&f)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 b = *(reinterpret_cast<const float4*>(bias) + q);
    f[4 * q] += b.x;
    f[4 * q + 1] += b.y;
    f[4 * q + 2] += b.z;
    f[4 * q + 3] += b.w;
  }
}

// A thread moves runs of its own row, so a warp's access touches 32 rows: with 32 bytes
// a thread it moves whole sectors; with 16, half of each twice. Rows that begin in the
// middle of a sector are moved as 16, 32 and 16 bytes (2751 x 1000 x 2056 with a
// residual and z: 29.0 us as four times 16, 28.3 so).
__device__ __forceinline__ void store_sector8(void* p, const uint32_t (&r)[8]) {
  store_sector(p, make_uint4(r[0], r[1], r[2], r[3]), make_uint4(r[4], r[5], r[6], r[7]));
}
__device__ __forceinline__ bool sector_aligned(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

// 32 columns of a residual row, as far as they exist (`left`, a multiple of 8).
struct Resid32 {
  uint4 v[4];
  template <int Q>
  __device__ __forceinline__ void one(const mf_bf16* p, int left) {
    if (left > 8 * Q) v[Q] = *(reinterpret_cast<const uint4*>(p) + Q);
  }
  template <int Q>
  __device__ __forceinline__ void two(const mf_bf16* p, int left) {
    if (left > 8 * Q + 8)
      load_sector(p + 8 * Q, v[Q], v[Q + 1]);
    else
      one<Q>(p, left);
  }
  __device__ __forceinline__ void load(const mf_bf16* p, int left) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = make_uint4(0, 0, 0, 0);
    if (sector_aligned(p)) {
      two<0>(p, left);
      two<2>(p, left);
    } else {
      one<0>(p, left);
      two<1>(p, left);
      one<3>(p, left);
    }
  }
  __device__ __forceinline__ void add(float (&f)[32]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float r[8];
      bf16x8_unpack(v[q], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[8 * q + e] += r[e];
    }
  }
};

// Up to 32 columns (`left`, a multiple of 8) in bf16.
__device__ __forceinline__ void store32(mf_bf16* p, int left, const float (&f)[32]) {
  uint4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    v[q] = make_uint4(pack_bf16x2(f[8 * q], f[8 * q + 1]), pack_bf16x2(f[8 * q + 2], f[8 * q + 3]),
                      pack_bf16x2(f[8 * q + 4], f[8 * q + 5]), pack_bf16x2(f[8 * q + 6], f[8 * q + 7]));
  auto one = [&](int q) {
    if (left > 8 * q) __stcs(reinterpret_cast<uint4*>(p) + q, v[q]);
  };
  auto two = [&](int q) {
    if (left > 8 * q + 8)
      store_sector(p + 8 * q, v[q], v[q + 1]);
    else
      one(q);
  };
  if (sector_aligned(p)) {
    two(0);
    two(2);
  } else {
    one(0);
    two(1);
    one(3);
  }
}

// Up to 32 codes.
__device__ __forceinline__ void store32_codes(int8_t* p, int left, const float (&f)[32], float inv,
                                              uint32_t mask) {
  uint32_t r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    r[e] = act8_code4(f2_pack(f[4 * e], f[4 * e + 1]), f2_pack(f[4 * e + 2], f[4 * e + 3]), inv, mask);
  if (left >= 32 && sector_aligned(p)) {
    store_sector8(p, r);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (left > 8 * q)
        __stcs(reinterpret_cast<uint2*>(p) + q, make_uint2(r[2 * q], r[2 * q + 1]));
  }
}

// The forward's epilogue on columns [cc0, cc1) of one row of a tile (a block of
// scales at most): bias, the kept pre-activation, activation, residual. With an
// 8-bit checkpoint the row's values of the block are read twice from TMEM, once for
// their largest magnitude; z itself never reaches memory. bias: the tile's, in shared
// memory, or NULL; res: the residual's first 32 columns, asked for before the
// accumulator was waited for (each next 32 are asked for one step ahead).
__device__ __forceinline__ void forward_row(const FwdArgs& a, uint32_t taddr, int t, bool keep,
                                            int n0, int cc0, int cc1, const float* bias,
                                            Resid32& res) {
  const LinearEpilogue& ep = a.ep;
  const size_t rowoff = static_cast<size_t>(t) * a.N;
  float s = 0.f, inv = 0.f;
  uint32_t mask = 0;
  if (ep.z8 != nullptr && cc0 < cc1) {
    uint32_t top = 0;
#pragma unroll 1
    for (int cc = cc0; cc < cc1; cc += 32) {
      float f[32];
      acc_load32(taddr + cc, f);
      if (bias != nullptr) add_bias32(bias + cc, f);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (e < cc1 - cc) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    }
    act8_scale(__uint_as_float(top), s, inv);
    mask = inv == 0.f ? 0u : 0xFFFFFFFFu;
    if (keep)
      ep.z_scale[static_cast<size_t>(t) * ((a.N + kAct8Block - 1) / kAct8Block) +
                 (n0 + cc0) / kAct8Block] = s;
  }
#pragma unroll 1
  for (int cc = cc0; cc < cc1; cc += 32) {
    const int c0 = n0 + cc, left = cc1 - cc;
    float f[32];
    Resid32 next;
    if (ep.resid != nullptr && keep) next.load(ep.resid + rowoff + c0 + 32, left - 32);
    acc_load32(taddr + cc, f);
    if (bias != nullptr) add_bias32(bias + cc, f);
    if (ep.z8 != nullptr && keep) store32_codes(ep.z8 + rowoff + c0, left, f, inv, mask);
    if (ep.z != nullptr && keep) store32(ep.z + rowoff + c0, left, f);
    if (ep.act == MF_ACT_GELU) act32<MF_ACT_GELU>(f);
    if (ep.act == MF_ACT_SILU) act32<MF_ACT_SILU>(f);
    if (keep) {
      if (ep.resid != nullptr) res.add(f);
      store32(ep.out + rowoff + c0, left, f);
    }
    res = next;
  }
}

// A pair's units, one of each round of `pairs`: in even rounds those of its own number
// and in odd ones from the other end, so that with the longest units first the pairs
// that had the longest get the shortest of what is left (dz, dx and dW of 1000 -> 2056
// over 2751 tokens: 51.3 -> 47.1 us; no difference where there are many rounds).
struct Queue {
  int u, even, odd;
  __device__ __forceinline__ Queue(int pair, int pairs)
      : u(pair), even(2 * pairs - 1 - 2 * pair), odd(2 * pair + 1) {}
  __device__ __forceinline__ void next() {
    u += even;
    const int t = even;
    even = odd;
    odd = t;
  }
};

// Maps: forward x, W; backward dz and W for dx, dz and x for dW (map_c, map_d).
template <int MODE>
__global__ void __launch_bounds__(kWarps * 32, 1)
    linear_fused_kernel(const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_b,
                        const __grid_constant__ CUtensorMap map_c,
                        const __grid_constant__ CUtensorMap map_d, int units,
                        const __grid_constant__ typename ArgsOf<MODE>::type args) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const int warp = warp_uniform(static_cast<int>(threadIdx.x) >> 5), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(&bars[i], i < kFull + kStages ? 2u : i == kAccEmpty || i == kAccEmpty + 1 ? 16u : 1u);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either reaches the other's
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*tmem_slot);
  pdl_wait();
  pdl_release();
  const int rank = warp_uniform(static_cast<int>(cluster_ctarank()));
  const Queue queue(static_cast<int>(blockIdx.x >> 1), static_cast<int>(gridDim.x >> 1));

  if (warp == 0) {
    // All lanes run the loop and lane 0 issues: with addresses and coordinates in uniform
    // registers the copies of a step are out in time for 0.22 us a step, like the MMAs
    // below (issued by one lane's branch: 0.29).
    const bool leader = lane == 0;
    const uint64_t keep = keep_in_l2();
    uint32_t it = 0, part_uses = 0;  // bit st: parity of PART[st]'s uses
    uint32_t part_used = 0;          // bit st: used at all
    bool ok = true;
    for (Queue q = queue; q.u < units && ok; q.next()) {
      const Unit w = unit_of(args, q.u);
      RunWalk walk;
      // this CTA's half of the tile's B columns; a strided B comes in boxes of 64
      int width;
      if constexpr (MODE == kFwd) {
        width = args.cols.width;
      } else {
        width = w.dw ? args.dw_cols.width : args.dx_cols.width;
        if (w.dw && w.steps > 0) walk.start(args, w);
      }
      const int half = width / 2;
      const bool two = half > 64;
      const uint32_t bytes =
          kABytes + (MODE == kFwd ? half * kStepK * 2 : two ? 2 * kBoxBytes : kBoxBytes);
      const int row = w.blk * kTile + rank * kHalf, col = w.ct * width + rank * half;
      for (int s = 0; s < w.steps; ++s, ++it) {
        const int st = it % kStages;
        if (!(ok = warp_wait(&bars[kEmpty + st], ((it / kStages) & 1) ^ 1, args.ctl, abort_flag)))
          break;
        uint8_t* sa = smem + st * kStageBytes;
        uint8_t* sb = sa + kABytes;
        if constexpr (MODE == kBwd) {
          if (w.dw) {
            if (walk.left < kStepK) {
              uint64_t* bar = &bars[kPart + st];
              expect_by(leader, bar, bytes);
              load_2d_by(leader, sa, &map_c, bar, row, walk.row);
              load_2d_by(leader, sa + kBoxBytes, &map_c, bar, row + 64, walk.row);
              load_2d_by(leader, sb, &map_d, bar, col, walk.row);
              if (two) load_2d_by(leader, sb + kBoxBytes, &map_d, bar, col + 64, walk.row);
              part_uses ^= 1u << st;
              part_used |= 1u << st;
            } else {
              const uint32_t bar = cluster_addr(&bars[kFull + st], 0);
              expect_pair(leader, bar, bytes);
              load_2d_pair_by(leader, sa, &map_c, bar, row, walk.row);
              load_2d_pair_by(leader, sa + kBoxBytes, &map_c, bar, row + 64, walk.row);
              load_2d_pair_by(leader, sb, &map_d, bar, col, walk.row);
              if (two) load_2d_pair_by(leader, sb + kBoxBytes, &map_d, bar, col + 64, walk.row);
            }
            walk.next(args, w.m);
            continue;
          }
        }
        const uint32_t bar = cluster_addr(&bars[kFull + st], 0);
        expect_pair(leader, bar, bytes);
        load_2d_pair_by(leader, sa, &map_a, bar, s * kStepK, row);
        if constexpr (MODE == kFwd) {
          load_w(leader, sb, &map_b, bar, s * kStepK, col, w.m, keep);
        } else {
          load_w(leader, sb, &map_b, bar, col, s * kStepK, w.m, keep);
          if (two) load_w(leader, sb + kBoxBytes, &map_b, bar, col + 64, s * kStepK, w.m, keep);
        }
      }
    }
    // Every copy lands before the CTA whose barrier it completes on can exit: the
    // leader waits for both CTAs' on FULL, each CTA for its own on PART.
    for (int st = 0; st < kStages; ++st) {
      if (rank == 0 && it > static_cast<uint32_t>(st)) {
        const uint32_t last = it - 1 - ((it - 1 - st) % kStages);
        drain_wait(&bars[kFull + st], (last / kStages) & 1, args.ctl.wait_limit_ns);
      }
      if ((part_used >> st) & 1)
        drain_wait(&bars[kPart + st], ((part_uses >> st) & 1) ^ 1, args.ctl.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // The leader CTA's warp: all lanes run the loop, lane 0 issues.
    if (rank == 0) {
      const bool leader = lane == 0;
      const uint32_t base = warp_uniform(smem_u32(smem));
      uint32_t it = 0, ul = 0;
      bool ok = true;
      // A unit's steps; DW and B_MN say which way the operands run. A contiguous inner
      // dimension: 16 elements are 32 bytes; a strided one: 16 rows of 128 bytes, the
      // 64-column boxes kBoxBytes apart.
      auto run = [&](auto dw, const Unit& w, uint32_t d, int width) {
        constexpr bool DW = decltype(dw)::value, B_MN = MODE == kBwd;
        constexpr uint64_t A_STEP = DW ? 128 : 2, B_STEP = B_MN ? 128 : 2;
        const uint64_t a_desc = sdesc_sw128(base, DW ? kBoxBytes : 16, 1024);
        const uint64_t b_desc = sdesc_sw128(base + kABytes, B_MN ? kBoxBytes : 16, 1024);
        const uint32_t idesc = idesc_bf16_f32(2 * kHalf, width, DW, B_MN);
        RunWalk walk;
        if constexpr (DW)
          if (w.steps > 0) walk.start(args, w);
        for (int s = 0; s < w.steps; ++s, ++it) {
          const int st = it % kStages;
          const uint32_t parity = (it / kStages) & 1;
          bool zeroed = false;  // rows zeroed by threads of both CTAs
          if constexpr (DW) {
            zeroed = walk.left < kStepK;
            walk.next(args, w.m);
          }
          ok = zeroed ? __all_sync(0xffffffffu, mbar_wait_cluster(&bars[kFull + st], parity,
                                                                  args.ctl, abort_flag))
                      : warp_wait(&bars[kFull + st], parity, args.ctl, abort_flag);
          if (!ok) return;
          tc_fence_after();
          const uint64_t so = static_cast<uint64_t>((st * kStageBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < kStepK / 16; ++kk)
            umma_ss_pair_by(leader, d, a_desc + so + kk * A_STEP, b_desc + so + kk * B_STEP, idesc,
                            (s > 0 || kk > 0) ? 1u : 0u);
          umma_commit_pair_by(leader, &bars[kEmpty + st], 3);
        }
      };
      for (Queue q = queue; q.u < units && ok; q.next(), ++ul) {
        const uint32_t acc = ul & 1;
        if (!warp_wait(&bars[kAccEmpty + acc], ((ul >> 1) & 1) ^ 1, args.ctl, abort_flag)) break;
        tc_fence_after();
        const Unit w = unit_of(args, q.u);
        const uint32_t d = tmem + acc * kTile;
        if constexpr (MODE == kFwd) {
          run(std::false_type{}, w, d, args.cols.width);
        } else {
          if (w.dw)
            run(std::true_type{}, w, d, args.dw_cols.width);
          else
            run(std::false_type{}, w, d, args.dx_cols.width);
        }
        if (!ok) break;
        umma_commit_pair_by(leader, &bars[kAccFull + acc], 3);
      }
      // every MMA this thread issued completes before TMEM is released
      umma_commit_pair_by(leader, &bars[kDrain], 1);
      drain_wait(&bars[kDrain], 0, args.ctl.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // A warp reaches the 32 TMEM lanes of its number modulo 4; warps 4..7 take the
    // tile's columns up to 128, warps 8..11 the rest.
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const int cc0 = warp >= 8 ? kTile / 2 : 0;
    uint32_t ul = 0;
    bool stop = false;  // a wait ran out: the forward's warps still meet at their barrier
    for (Queue q = queue; q.u < units; q.next(), ++ul) {
      const uint32_t acc = ul & 1;
      const uint32_t taddr = tmem + lane_base + acc * kTile;
      const Unit w = unit_of(args, q.u);
      const int r = w.blk * kTile + rank * kHalf + row;  // token, or row of dW
      if constexpr (MODE == kFwd) {
        const int n0 = w.ct * args.cols.width;
        const bool keep = r < args.T && __ldg(args.tok_mod + r) == w.m;
        const int end = min(min(cc0 + kTile / 2, args.cols.width), args.N - n0);
        float* bias = reinterpret_cast<float*>(smem + kOffBias);
        Resid32 res;
        if (args.ep.resid != nullptr && keep && cc0 < end)
          res.load(args.ep.resid + static_cast<size_t>(r) * args.N + n0 + cc0, end - cc0);
        if (args.ep.bias != nullptr) {
          const int c = static_cast<int>(threadIdx.x) - 4 * 32;
          const float v = n0 + c < args.N
                              ? __ldg(args.ep.bias + static_cast<size_t>(w.m) * args.N + n0 + c)
                              : 0.f;
          epilogue_sync();  // every warp is done with the tile before
          bias[c] = v;
          epilogue_sync();
        }
        if (!warp_wait(&bars[kAccFull + acc], (ul >> 1) & 1, args.ctl, abort_flag)) stop = true;
        tc_fence_after();
        if (!stop)
          forward_row(args, taddr, r, keep, n0, cc0, end, args.ep.bias != nullptr ? bias : nullptr,
                      res);
      } else {
        const int width = w.dw ? args.dw_cols.width : args.dx_cols.width;
        const int k0 = w.ct * width;
        const int end = min(min(cc0 + kTile / 2, width), args.K - k0);
        bool keep;
        mf_bf16* out;
        float* part = nullptr;
        if (w.dw) {
          keep = r < args.N;
          out = args.dW + (static_cast<size_t>(w.m) * args.N + r) * args.K + k0;
          if (w.slot >= 0)
            part = args.part +
                   (static_cast<size_t>(w.slot) * kTile + rank * kHalf + row) * kTile;
        } else {
          keep = r < args.T && __ldg(args.tok_mod + r) == w.m;
          out = args.dx + static_cast<size_t>(r) * args.K + k0;
        }
        if (!warp_wait(&bars[kAccFull + acc], (ul >> 1) & 1, args.ctl, abort_flag)) break;
        tc_fence_after();
#pragma unroll 1
        for (int cc = cc0; cc < end; cc += 32) {
          float f[32];
          acc_load32(taddr + cc, f);
          if (w.steps == 0)  // dW of a modality without tokens
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
          if (part != nullptr) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(f[8 * q + e]);
              store_sector8(part + cc + 8 * q, v);
            }
          } else if (keep) {
            store32(out + cc, end - cc, f);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&bars[kAccEmpty + acc], 0));
    }
  } else if (MODE == kBwd && warp == 3) {
    if constexpr (MODE == kBwd) {
      if (args.db.out != nullptr) {
        for (int c = static_cast<int>(blockIdx.x) * 32 + lane; c < args.db.cols;
             c += static_cast<int>(gridDim.x) * 32) {
          float v = 0.f;
#pragma unroll 8
          for (int k = 0; k < args.db.n; ++k)
            v += __ldcg(args.db.part + static_cast<size_t>(k) * args.db.cols + c);
          args.db.out[c] = v;
        }
      }
    }
  } else if (MODE == kBwd && warp == 2) {
    if constexpr (MODE == kBwd) {
      uint32_t it = 0, part_uses = 0;
      bool ok = true;
      for (Queue q = queue; q.u < units && ok; q.next()) {
        const Unit w = unit_of(args, q.u);
        if (!w.dw) {
          it += w.steps;
          continue;
        }
        if (w.steps == 0) continue;
        RunWalk walk;
        walk.start(args, w);
        for (int s = 0; s < w.steps; ++s, ++it, walk.next(args, w.m)) {
          const int live = walk.left;
          if (live >= kStepK) continue;
          const int st = it % kStages;
          if (!(ok = warp_wait(&bars[kPart + st], (part_uses >> st) & 1, args.ctl, abort_flag))) break;
          part_uses ^= 1u << st;
          // rows past the run in the four 64-column boxes: 128 bytes a row
          const int dead = (kStepK - live) * 8;
          uint8_t* sa = smem + st * kStageBytes + live * 128;
          for (int i = lane; i < dead; i += 32)
#pragma unroll
            for (int b = 0; b < 4; ++b)
              *reinterpret_cast<uint4*>(sa + b * kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();  // this thread's writes before the tensor core's reads
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&bars[kFull + st], 0));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Neither CTA frees TMEM or leaves before both are here: the leader's MMAs write
  // both CTAs' TMEM, and copies and arrivals cross between them.
  cluster_sync();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// dW[m] = the sum of its parts, in order, rounded once. One thread per 8 columns.
__global__ void __launch_bounds__(256) dw_parts_kernel(const float* __restrict__ part, int splits,
                                                       int N, int K, int width, int col_tiles,
                                                       int tiles, mf_bf16* __restrict__ dW) {
  pdl_wait();
  pdl_release();
  const int groups = K / 8;
  const int64_t total = static_cast<int64_t>(N) * groups;
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i < total) {
    const int n = static_cast<int>(i / groups), k = static_cast<int>(i - static_cast<int64_t>(n) * groups) * 8;
    const float* p = part + ((static_cast<size_t>(n / kTile) * col_tiles + k / width) * kTile +
                             n % kTile) * kTile + k % width;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s, p += static_cast<size_t>(tiles) * kTile * kTile) {
      const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
      f[0] += a.x; f[1] += a.y; f[2] += a.z; f[3] += a.w;
      f[4] += b.x; f[5] += b.y; f[6] += b.z; f[7] += b.w;
    }
    *reinterpret_cast<uint4*>(dW + static_cast<size_t>(n) * K + k) = bf16x8_pack(f);
  }
}

// ------------------------------------------------------------ dz and db
// dz = dout act'(z) and the modality sums of the unrounded dz. dz is rounded to bf16, the
// type of both products' operands (as an 8-bit x is, below): operands of twice the bits run
// at half the rate or less, and dW's relative RMS, 1.7e-3 from its own rounding to bf16,
// becomes 2.3e-3 with one operand rounded and 2.9e-3 with both.
// A CTA takes `rows` rows of 256 channels: 32 lanes of eight channels by eight row lanes,
// four rows of loads in flight per thread; the row lanes' sums meet in shared memory and
// leave as part[chunk][modality][N], which a warp of the next product's kernel adds in
// order (or db itself, when one chunk holds every row). HBM-bound. ACT none: only the
// sums. The blocks behind these decode an 8-bit x for dW: one launch for both.
constexpr int kDzUnroll = 4;

// Short packs get short chunks, so that there are CTAs for every SM.
int dz_rows(int32_t T) { return T <= 2048 ? 32 : T <= 8192 ? 64 : 128; }
int dz_chunks(int32_t T) { return (T + dz_rows(T) - 1) / dz_rows(T); }
// The most chunks of any pack of up to T tokens: what the workspace is sized by, so that
// one taken for a long pack serves shorter ones.
int dz_chunks_most(int32_t T) {
  const int least = T <= 2048 ? 0 : dz_chunks(T <= 8192 ? 2048 : 8192);
  return dz_chunks(T) > least ? dz_chunks(T) : least;
}

struct Decode {
  Act8 x8;
  Act8Rows rows;  // no items: nothing to decode
  mf_bf16* y;
  bool wide;
};

template <int ACT, bool Z8>
__global__ void __launch_bounds__(256) dz_kernel(const mf_bf16* __restrict__ dout,
                                                 const mf_bf16* __restrict__ z, const Act8 z8,
                                                 const uint8_t* __restrict__ tok_mod, int T, int N,
                                                 int rows, int col_blocks, int dz_blocks,
                                                 mf_bf16* __restrict__ dz, float* __restrict__ part,
                                                 const Decode dec, KernelCtl ctl) {
  __shared__ float acc[2][8][256];
  pdl_wait();
  pdl_release();
  if (static_cast<int>(blockIdx.x) >= dz_blocks) {
    if (dec.wide)
      act8_decode<MF_ACT_NONE, true>(dec.x8.q, dec.x8.scale, dec.rows, dec.y, blockIdx.x - dz_blocks);
    else
      act8_decode<MF_ACT_NONE, false>(dec.x8.q, dec.x8.scale, dec.rows, dec.y, blockIdx.x - dz_blocks);
    return;
  }
  const int chunk = blockIdx.x / col_blocks, cb = blockIdx.x - chunk * col_blocks;
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int c = cb * 256 + cl * 8;
  const bool on = c < N;
  const int nb = (N + kAct8Block - 1) / kAct8Block;
  const int r0 = chunk * rows, r1 = min(T, r0 + rows);
  uint64_t sum[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[0][e] = sum[1][e] = 0;
  for (int t0 = r0 + rl; t0 < r1; t0 += 8 * kDzUnroll) {
    uint4 vd[kDzUnroll], vz[kDzUnroll];
    float vs[kDzUnroll];
    int mod[kDzUnroll];
#pragma unroll
    for (int u = 0; u < kDzUnroll; ++u) {
      const int t = t0 + u * 8;
      const bool live = t < r1 && on;
      const size_t off = static_cast<size_t>(t) * N + c;
      mod[u] = live ? __ldg(tok_mod + t) : 2;
      vd[u] = live ? __ldg(reinterpret_cast<const uint4*>(dout + off)) : make_uint4(0, 0, 0, 0);
      vz[u] = make_uint4(0, 0, 0, 0);
      vs[u] = 0.f;
      if (ACT != MF_ACT_NONE && live) {
        if constexpr (Z8) {
          const uint2 q = __ldcs(reinterpret_cast<const uint2*>(z8.q + off));
          vz[u].x = q.x;
          vz[u].y = q.y;
          vs[u] = __ldg(z8.scale + static_cast<size_t>(t) * nb + c / kAct8Block);
        } else {
          vz[u] = __ldcs(reinterpret_cast<const uint4*>(z + off));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kDzUnroll; ++u) {
      const int t = t0 + u * 8;
      if (t >= r1 || !on) continue;
      uint64_t d[4];
      bf16x8_f2(vd[u], d);
      if constexpr (ACT != MF_ACT_NONE) {
        uint64_t f[4];
        if constexpr (Z8)
          act8_load(make_uint2(vz[u].x, vz[u].y), vs[u], f);
        else
          bf16x8_f2(vz[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = f2_mul(d[e], act_grad2<ACT>(f[e]));
        *reinterpret_cast<uint4*>(dz + static_cast<size_t>(t) * N + c) = f2_bf16x8(d);
      }
      if (mod[u] > 1) {
        atomicCAS(ctl.err, 0, static_cast<int>(MF_ERR_INVALID));
        continue;
      }
      if (mod[u] == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[0][e] = f2_add(sum[0][e], d[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[1][e] = f2_add(sum[1][e], d[e]);
      }
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f2_unpack(sum[m][e], acc[m][rl][cl * 8 + 2 * e], acc[m][rl][cl * 8 + 2 * e + 1]);
  __syncthreads();
  const int col = cb * 256 + threadIdx.x;
  if (col < N) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) v += acc[m][r][threadIdx.x];
      part[(static_cast<size_t>(chunk) * 2 + m) * N + col] = v;
    }
  }
}

// db's partials where no product follows: one thread per column.
__global__ void __launch_bounds__(128) dz_cols_kernel(const ColumnSums db) {
  pdl_wait();
  pdl_release();
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (c >= db.cols) return;
  float v = 0.f;
#pragma unroll 8
  for (int k = 0; k < db.n; ++k) v += __ldcg(db.part + static_cast<size_t>(k) * db.cols + c);
  db.out[c] = v;
}

// ------------------------------------------------------------ host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                       cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p)
               : nullptr;
  }();
  return fn;
}

template <int MODE>
cudaLaunchConfig_t config(int clusters, cudaLaunchAttribute* attr, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of two that can be resident at once; 0 if the kernel cannot run.
template <int MODE>
int max_clusters() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cached[dev] == 0) {
    if (cudaFuncSetAttribute(linear_fused_kernel<MODE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes) != cudaSuccess)
      return 0;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config<MODE>(1, attr, nullptr);
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, linear_fused_kernel<MODE>, &cfg) != cudaSuccess)
      return 0;
    cached[dev] = n;
  }
  return cached[dev];
}

template <int MODE>
cudaError_t launch_product(const CUtensorMap (&m)[4], const typename ArgsOf<MODE>::type& a,
                           int units, cudaStream_t st) {
  const int mc = max_clusters<MODE>();
  if (mc <= 0) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config<MODE>(units < mc ? units : mc, attr, st);
  return cudaLaunchKernelEx(&cfg, linear_fused_kernel<MODE>, m[0], m[1], m[2], m[3], units, a);
}

int tiles_of(int64_t v) { return static_cast<int>((v + kTile - 1) / kTile); }

// Row blocks of kTile rows and the modalities each holds; T <= kMaxGemmTiles * 128.
void row_jobs(const TokenRuns& runs, int32_t T, GemmJobs* jobs) {
  static thread_local uint8_t has[kMaxGemmTiles];
  const int tiles = tiles_of(T);
  memset(has, 0, static_cast<size_t>(tiles));
  for (int m = 0; m < 2; ++m)
    for (int r = 0; r < runs.n[m]; ++r)
      for (int b = runs.start[m][r] / kTile; b <= (runs.start[m][r] + runs.len[m][r] - 1) / kTile; ++b)
        has[b] |= 1u << m;
  jobs->n = 0;
  for (int b = 0; b < tiles; ++b)
    for (int m = 0; m < 2; ++m)
      if (has[b] & (1u << m)) jobs->job[jobs->n++] = static_cast<uint16_t>(b | (m << 15));
}

// Width of the column tiles: 256, or 128 or 64 while all tiles then still fit one
// round over the pairs of SMs (short packs, small layers: the epilogue, which no next
// tile's MMAs hide there, shrinks with the width).
int tile_width(int rows, int cols, int pairs, int least) {
  int w = kTile;
  while (w / 2 >= least && rows * ((cols + w / 2 - 1) / (w / 2)) <= pairs) w /= 2;
  return w;
}

// The forward's, in two or three rounds: the width whose rounds cost least, a round
// as much as its width and 200 columns more (1000 -> 2056 over 2751 tokens: 208
// columns, 22.2 us against 24.0; 1024 -> 4096 over 2464: 192, 24.1 against 26.2).
// Beyond that 256 is best whatever the last round holds (8464 x 3072 x 12288: 240
// columns would be 22.5 rounds' worth in place of 23 and take 429 us in place of 421),
// and dx, whose B operand comes in 64-column boxes, loses at widths between them
// (4096 -> 1024 over 2464: 30.8 us at 240 against 27.9).
int forward_width(int rows, int cols, int pairs, bool blocks) {
  const int w = tile_width(rows, cols, pairs, blocks ? kAct8Block : 64);
  if (w < kTile || blocks || pairs <= 0) return w;
  int best = w, cost = 0;
  for (int v = kTile; v >= 128; v -= 16) {
    const int rounds = (rows * ((cols + v - 1) / v) + pairs - 1) / pairs;
    if (v == kTile && rounds > 3) return kTile;
    if (v == kTile || rounds * (v + 200) < cost) {
      best = v;
      cost = rounds * (v + 200);
    }
  }
  return best;
}

Columns columns(int cols, int width) {
  while (width > 64 && width / 2 >= cols) width /= 2;  // no wider than the output
  const int tiles = (cols + width - 1) / width;
  return Columns{width, tiles, tiles < 12 ? tiles : 12};
}

// Pairs of SMs on a B200 (148 SMs): what dW's split and its workspace are sized by.
constexpr int kPairs = 74;

// Tiles of one modality's dW at a column width.
int dw_tiles(int32_t K, int32_t N, int width) {
  return tiles_of(N) * ((K + width - 1) / width);
}

// Parts of a modality's steps: as many as fill the pairs, of at least kDwPartSteps
// steps each, if that takes at least kDwJoinSteps steps off: a step takes about
// 0.33 us, joining the parts about 8 us (dx and dW, 256 -> 1024 over 4160 tokens: 20.4
// us in 2 parts, 16.0 in 5; 1000 -> 2056 over 2751: 43.2 in 2 parts, 40.2 whole).
constexpr int kDwPartSteps = 12, kDwJoinSteps = 24;
int dw_splits(int tiles, int steps) {
  const int by_pairs = kPairs / tiles, by_steps = steps / kDwPartSteps;
  const int p = by_pairs < by_steps ? by_pairs : by_steps;
  return p > 1 && steps - (steps + p - 1) / p >= kDwJoinSteps ? p : 1;
}

// The most steps that one modality of a pack of T tokens can have: a run ends in at most
// one step that it does not fill, and a token of the other modality at least lies between
// two runs.
int dw_steps_most(int32_t T) {
  const int32_t runs = (T + 1) / 2;
  return T / kStepK + (runs < MF_MAX_SAMPLES ? runs : MF_MAX_SAMPLES);
}

// Column width of dW's tiles: 256 if a modality's steps are split, and otherwise
// narrower only while its tiles and the launch's others (`sets` modalities, `dx`) fit
// one round: a step takes as long at any width, so narrow tiles in several rounds lose
// (dx and dW, 512 -> 2048 over 8464 tokens: 57.2 us at 64 columns, 36.4 at 256 in
// parts; 1000 -> 1000 over 3912: 37.5 and 31.8).
int dw_width(int32_t K, int32_t N, const int steps[2], int dx) {
  int w = kTile;
  const int tiles = dw_tiles(K, N, w), sets = (steps[0] > 0) + (steps[1] > 0);
  if (dw_splits(tiles, steps[0]) > 1 || dw_splits(tiles, steps[1]) > 1) return w;
  while (w > 64 && dx + sets * dw_tiles(K, N, w / 2) <= kPairs) w /= 2;
  return w;
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

bool linear_map(CUtensorMap* map, const mf_bf16* base, int64_t cols, int64_t rows, int sets,
                int box_rows) {
  const EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(sets)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols * 2),
                                 static_cast<cuuint64_t>(cols * rows * 2)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, sets > 0 ? 3 : 2, const_cast<mf_bf16*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool token_runs(const mf_sample_desc* desc, int32_t S, TokenRuns* runs, int32_t* T) {
  memset(runs->n, 0, sizeof(runs->n));
  memset(runs->count, 0, sizeof(runs->count));
  int64_t row = 0;
  for (int32_t s = 0; s < S; ++s) {
    const mf_sample_desc& d = desc[s];
    if (d.frames < 0 || d.grid_h < 0 || d.grid_w < 0 || d.n_text < 0 || d.grid_h > MF_MAX_TOKENS ||
        d.grid_w > MF_MAX_TOKENS || d.frames > MF_MAX_TOKENS)
      return false;
    const int64_t plane = static_cast<int64_t>(d.grid_h) * d.grid_w;
    if (plane > MF_MAX_TOKENS) return false;
    const int64_t n[2] = {d.frames * plane, d.n_text};
    for (int m = 0; m < 2; ++m) {
      if (row + n[m] > MF_MAX_TOKENS) return false;
      if (n[m] == 0) continue;
      const int r = runs->n[m];
      if (r > 0 && runs->start[m][r - 1] + runs->len[m][r - 1] == row) {
        runs->len[m][r - 1] += static_cast<int32_t>(n[m]);
      } else {
        runs->start[m][r] = static_cast<int32_t>(row);
        runs->len[m][r] = static_cast<int32_t>(n[m]);
        runs->n[m] = r + 1;
      }
      runs->count[m] += static_cast<int32_t>(n[m]);
      row += n[m];
    }
  }
  *T = static_cast<int32_t>(row);
  return true;
}

cudaError_t launch_linear_fused(const mf_bf16* x, const mf_bf16* W, const TokenRuns& runs,
                                const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                                const LinearEpilogue& ep, const KernelCtl& ctl, cudaStream_t st) {
  if (few_rows(T)) return launch_linear_rows(x, W, runs, tok_mod, T, K, N, ep, ctl, st);
  static thread_local FwdArgs a;
  row_jobs(runs, T, &a.jobs);
  a.T = T;
  a.K = K;
  a.N = N;
  a.cols = columns(N, forward_width(a.jobs.n, N, max_clusters<kFwd>(), ep.z8 != nullptr));
  a.tok_mod = tok_mod;
  a.ep = ep;
  a.ctl = ctl;
  CUtensorMap m[4];
  if (!linear_map(&m[0], x, K, T, 0, kHalf) ||
      !linear_map(&m[1], W, K, N, 2, a.cols.width / 2))
    return cudaErrorInvalidValue;
  m[2] = m[3] = m[0];
  return launch_product<kFwd>(m, a, a.jobs.n * a.cols.tiles, st);
}

// Workspace, in this order: dz [T][N] bf16; db's partials; an 8-bit x in bf16; dW's
// parts.
size_t linear_fused_bwd_ws(int32_t T, int32_t K, int32_t N) {
  const size_t chunks = dz_chunks_most(T);
  const int tiles = dw_tiles(K, N, kTile), splits = dw_splits(tiles, dw_steps_most(T));
  const size_t parts = splits > 1 ? static_cast<size_t>(2) * tiles * splits : 0;
  return round256(static_cast<size_t>(T) * N * 2) + round256(chunks * 2 * N * sizeof(float)) +
         round256(static_cast<size_t>(T) * K * 2) + parts * kTile * kTile * sizeof(float);
}

cudaError_t launch_linear_fused_bwd(const LinearBwd& b, const TokenRuns& runs, int32_t T, int32_t K,
                                    int32_t N, void* ws, const KernelCtl& ctl, cudaStream_t st) {
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  mf_bf16* dz_ws = reinterpret_cast<mf_bf16*>(w);
  w += round256(static_cast<size_t>(T) * N * 2);
  const int rows = dz_rows(T), chunks = dz_chunks(T);
  float* part = reinterpret_cast<float*>(w);
  w += round256(static_cast<size_t>(chunks) * 2 * N * sizeof(float));
  mf_bf16* x_ws = reinterpret_cast<mf_bf16*>(w);
  w += round256(static_cast<size_t>(T) * K * 2);
  float* dw_part = reinterpret_cast<float*>(w);
  cudaError_t e;

  const mf_bf16* dz = b.act == MF_ACT_NONE ? b.dout : dz_ws;
  ColumnSums db = {part, chunks, 2 * N, chunks > 1 ? b.db : nullptr};
  // An 8-bit x is decoded once into the workspace (3 bytes of traffic a value, a
  // tenth of the product's time at 8464 x 12288 x 3072); decoding it between the
  // copies and the MMAs, again for every 256 output rows, took 2.6 times as long
  // as the product.
  Decode dec = {};
  if (b.dW != nullptr && b.x == nullptr)
    dec = Decode{b.x8, act8_rows(T, K), x_ws, act8_wide(x_ws, K)};  // T blocks <= 2^17 2^13: below 2^31
  const int col_blocks = (N + 255) / 256;
  const int dz_blocks = b.act != MF_ACT_NONE || b.db != nullptr ? chunks * col_blocks : 0;
  const unsigned blocks = dz_blocks + act8_ctas(dec.rows.items, dec.wide);
  if (blocks > 0) {
    float* p = b.db == nullptr ? nullptr : chunks > 1 ? part : b.db;
#define MF_DZ(ACT, Z8)                                                                           \
  launch_dependent(dz_kernel<ACT, Z8>, dim3(blocks), dim3(256), 0, st, b.dout, b.z, b.z8,        \
                   b.tok_mod, T, N, rows, col_blocks, dz_blocks, dz_ws, p, dec, ctl)
    if (b.act == MF_ACT_NONE) e = MF_DZ(MF_ACT_NONE, false);
    else if (b.act == MF_ACT_GELU && b.z8.q != nullptr) e = MF_DZ(MF_ACT_GELU, true);
    else if (b.act == MF_ACT_GELU) e = MF_DZ(MF_ACT_GELU, false);
    else if (b.z8.q != nullptr) e = MF_DZ(MF_ACT_SILU, true);
    else e = MF_DZ(MF_ACT_SILU, false);
#undef MF_DZ
    if (e != cudaSuccess) return e;
  }

  const bool few_dx = b.dx != nullptr && few_rows(T);
  if (few_dx) {
    e = launch_linear_rows_dx(dz, b.W, runs, b.tok_mod, T, K, N, b.dx, ctl, st);
    if (e != cudaSuccess) return e;
  }
  if ((b.dx != nullptr && !few_dx) || b.dW != nullptr) {
    static thread_local BwdArgs a;
    a.T = T;
    a.K = K;
    a.N = N;
    a.tok_mod = b.tok_mod;
    a.dx = b.dx;
    a.dW = b.dW;
    a.part = dw_part;
    a.db = db;
    a.ctl = ctl;
    db.out = nullptr;
    CUtensorMap m[4];
    int units[3] = {0, 0, 0};
    int64_t cost[3] = {0, 0, 0};  // of a unit, by kind
    a.jobs.n = 0;
    a.dx_cols = a.dw_cols = columns(K, kTile);
    if (b.dx != nullptr && !few_dx) {
      if (!linear_map(&m[0], dz, N, T, 0, kHalf) || !linear_map(&m[1], b.W, K, N, 2, kStepK))
        return cudaErrorInvalidValue;
      row_jobs(runs, T, &a.jobs);
      // narrower tiles where they fill SMs that nothing else would
      a.dx_cols = columns(
          K, b.dW != nullptr ? kTile : tile_width(a.jobs.n, K, max_clusters<kBwd>(), 64));
      units[kDx] = a.jobs.n * a.dx_cols.tiles;
      cost[kDx] = static_cast<int64_t>((N + kStepK - 1) / kStepK) * a.dx_cols.width;
    }
    int slots = 0;
    if (b.dW != nullptr) {
      if (!linear_map(&m[2], dz, N, T, 0, kStepK) ||
          !linear_map(&m[3], b.x != nullptr ? b.x : x_ws, K, T, 0, kStepK))
        return cudaErrorInvalidValue;
      for (int i = 0; i < 2; ++i) {
        a.n[i] = runs.n[i];
        a.it0[i][0] = 0;
        for (int r = 0; r < runs.n[i]; ++r) {
          a.start[i][r] = runs.start[i][r];
          a.len[i][r] = runs.len[i][r];
          a.it0[i][r + 1] = a.it0[i][r] + (runs.len[i][r] + kStepK - 1) / kStepK;
        }
      }
      const int steps[2] = {a.it0[0][runs.n[0]], a.it0[1][runs.n[1]]};
      a.dw_cols = columns(K, dw_width(K, N, steps, units[kDx]));
      const int tiles = tiles_of(N) * a.dw_cols.tiles;
      for (int i = 0; i < 2; ++i) {
        a.splits[i] = dw_splits(tiles, steps[i]);
        a.slot0[i] = slots;
        units[kDwImage + i] = tiles * a.splits[i];
        if (a.splits[i] > 1) slots += units[kDwImage + i];
        cost[kDwImage + i] = static_cast<int64_t>(steps[i] / a.splits[i]) * a.dw_cols.width;
      }
    }
    if (b.dx == nullptr || few_dx) m[0] = m[1] = m[2];
    if (b.dW == nullptr) m[2] = m[3] = m[0];
    // the queue: the kind with the longest units first
    int total = 0;
    bool queued[3] = {false, false, false};
    for (int q = 0; q < 3; ++q) {
      int best = -1;
      for (int k = 0; k < 3; ++k)
        if (!queued[k] && (best < 0 || cost[k] > cost[best])) best = k;
      queued[best] = true;
      a.kind[q] = best;
      a.end[q] = total += units[best];
    }
    e = launch_product<kBwd>(m, a, total, st);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < 2 && b.dW != nullptr; ++i) {
      if (a.splits[i] == 1) continue;
      const int64_t groups = static_cast<int64_t>(N) * (K / 8);
      e = launch_dependent(dw_parts_kernel, dim3(static_cast<unsigned>((groups + 255) / 256)),
                           dim3(256), 0, st,
                           dw_part + static_cast<size_t>(a.slot0[i]) * kTile * kTile, a.splits[i],
                           N, K, a.dw_cols.width, a.dw_cols.tiles,
                           tiles_of(N) * a.dw_cols.tiles, b.dW + static_cast<size_t>(i) * N * K);
      if (e != cudaSuccess) return e;
    }
  }
  if (db.out != nullptr)
    return launch_dependent(dz_cols_kernel, dim3((db.cols + 127) / 128), dim3(128), 0, st, db);
  return cudaSuccess;
}

}  // namespace mf
