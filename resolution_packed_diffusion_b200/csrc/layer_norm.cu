// layer_norm.cu -- the modality-specific layer norm with weights and its backward:
//   y = (x - mean) rstd gamma[m] + beta[m], m the token's modality (0 image, 1 text);
//   g = dy gamma[m], xhat = (x - mean) rstd,
//   dx = resid + rstd (g - mean(g) - xhat mean(g xhat)),
//   dgamma[m] = sum of dy xhat, dbeta[m] = sum of dy over the modality's tokens.
// Source (page title, section): picx.dev "Mage-Flow" summary, Methodology >
// Native-Resolution MMDiT (each stream keeps its own normalization).
//
// Both passes are bound by HBM: the forward reads and writes a row once, the
// backward reads x (bf16, or an 8-bit checkpoint of it), dy and resid once and
// writes dx.
//
// Forward, rows of 264 to 4096 channels (layer_norm_rows_kernel): a warp per row,
// the row in registers for the mean, the variance about the mean (no cancellation)
// and the output; one persistent CTA per SM, so that gamma and beta of both
// modalities are read from shared memory and not once more per row from L1 or L2.
// Narrower and wider rows (layer_norm_kernel): a row is shared by a group of threads
// (8, 16 or 32 lanes, or several warps), a thread owning eight channels whose gamma
// and beta stay in registers; R rows per step, the next step's loads in flight.
//
// Backward: column ownership as there, since a thread then also keeps its channels'
// running dgamma and dbeta in registers. A step's rows lie next to each other, so
// one bulk copy per tensor brings them into a ring of shared-memory stages; the row
// sums of g and g xhat are reduced by shuffles and, over several warps, at the one
// barrier a step has, after which dx is formed from the same stage. The column sums
// leave the registers when the modality changes, to the group's own place, and at the
// end; the CTAs of a cluster add theirs over distributed shared memory, and a second
// kernel adds the clusters' in a fixed order: no atomics, the same bits every time.
#include <cuda_bf16.h>

#include <cstdint>

#include "act8.cuh"
#include "linear_common.cuh"
#include "mlp_internal.h"
#include "pdl.cuh"

namespace mf {

namespace {

int ln_sms() {
  static int cached[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

// How a CTA's threads share rows: groups of `lanes` threads (a power of two up
// to 32, or whole warps), one 8-channel chunk per thread.
struct RowShape {
  int lanes;    // threads of a group
  int groups;   // groups of a CTA
  int threads;
};

RowShape row_shape(int32_t hid) {
  const int chunks = hid / 8;
  RowShape s;
  if (chunks <= 32) {
    s.lanes = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    s.groups = 256 / s.lanes;
  } else {
    s.lanes = (chunks + 31) / 32 * 32;
    s.groups = s.lanes >= 256 ? 1 : 256 / s.lanes;
  }
  s.threads = s.lanes * s.groups;
  return s;
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums v[0..NV) over the group. SUB lanes by shuffles; with W > 1 warps the
// warps' sums meet in shared memory (two buffers, so one barrier per call).
template <int NV, int SUB>
__device__ __forceinline__ void group_sum(float (&v)[NV], int warps, int group, int warp_in_group,
                                          float* red, int& flip) {
#pragma unroll
  for (int o = SUB / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (SUB == 32 && warps > 1) {
    // red: [2][groups * warps][8], NV <= 8
    float* buf = red + (flip * 32 + group * warps) * 8;
    flip ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) buf[warp_in_group * 8 + i] = v[i];
    }
    named_barrier(1 + group, warps * 32);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] += buf[w * 8 + i];
  }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p + 4));
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void load8_f2(const float* p, uint64_t (&f)[4]) {
  const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p));
  const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

struct LnArgs {
  const uint8_t* tok_mod;
  int T, hid, lanes, groups;
  KernelCtl ctl;
};

// The rows of this CTA: contiguous, in whole steps of groups * R rows.
template <int R>
__device__ __forceinline__ void cta_rows(const LnArgs& a, int& r0, int& r1) {
  const int step = a.groups * R;
  const int steps = (a.T + step - 1) / step;
  const int per = (steps + gridDim.x - 1) / gridDim.x;
  r0 = min(a.T, static_cast<int>(blockIdx.x) * per * step);
  r1 = min(a.T, r0 + per * step);
}

template <int SUB, int R, int THREADS>
__global__ void __launch_bounds__(THREADS) layer_norm_kernel(const mf_bf16* __restrict__ x,
                                                             const float* __restrict__ gamma,
                                                             const float* __restrict__ beta,
                                                             const LnArgs a, float eps,
                                                             mf_bf16* __restrict__ y,
                                                             float2* __restrict__ stats) {
  __shared__ float red[2 * 32 * 8];
  const int group = threadIdx.x / a.lanes, gl = threadIdx.x - group * a.lanes;
  const int warps = a.lanes / 32, wig = gl / 32;
  const int c = gl * 8;
  const bool on = c < a.hid;
  const float inv_n = 1.f / static_cast<float>(a.hid);
  int r0, r1, flip = 0;
  cta_rows<R>(a, r0, r1);
  float gam[8], bet[8];
  int cm = -1;
  pdl_wait();
  pdl_release();
  uint4 next[R];
  int mod_next[R];
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool live = row + i < r1;
      mod_next[i] = live ? __ldg(a.tok_mod + row + i) : -1;
      next[i] = live && on ? __ldcs(reinterpret_cast<const uint4*>(
                                 x + static_cast<size_t>(row + i) * a.hid + c))
                           : make_uint4(0, 0, 0, 0);
    }
  };
  const int step = a.groups * R;
  fetch(r0 + group * R);
  // every group of the CTA takes the same number of steps: its rows past the end
  // are not live, but its lanes shuffle with their warp's other groups
  for (int base = r0; base < r1; base += step) {
    const int row = base + group * R;
    uint4 v[R];
    int mod[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      v[i] = next[i];
      mod[i] = mod_next[i];
    }
    fetch(row + step);
    float mean[R], var[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float f[8];
      bf16x8_unpack(v[i], f);
      mean[i] = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
    }
    group_sum<R, SUB>(mean, warps, group, wig, red, flip);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      mean[i] *= inv_n;
      float f[8], s = 0.f;
      bf16x8_unpack(v[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = f[e] - mean[i];
        s = fmaf(d, d, s);
      }
      var[i] = on ? s : 0.f;
    }
    group_sum<R, SUB>(var, warps, group, wig, red, flip);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (mod[i] < 0) continue;
      if (mod[i] > 1) {
        if (gl == 0) atomicCAS(a.ctl.err, 0, static_cast<int>(MF_ERR_INVALID));
        continue;
      }
      const float rstd = rsqrtf(fmaf(var[i], inv_n, eps));
      if (mod[i] != cm) {
        cm = mod[i];
        if (on) {
          load8(gamma + static_cast<size_t>(cm) * a.hid + c, gam);
          load8(beta + static_cast<size_t>(cm) * a.hid + c, bet);
        }
      }
      if (on) {
        float f[8];
        bf16x8_unpack(v[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean[i]) * rstd, gam[e], bet[e]);
        __stcs(reinterpret_cast<uint4*>(y + static_cast<size_t>(row + i) * a.hid + c),
               bf16x8_pack(f));
      }
      if (gl == 0 && stats != nullptr) stats[row + i] = make_float2(mean[i], rstd);
    }
  }
}

// One warp per row of NCH x 256 channels at most. Dynamic shared memory:
// [2 modalities][gamma, beta][2][hid / 8] float4, the first and the second four of
// every eight channels apart, so that a warp's reads meet no bank twice.
__device__ __forceinline__ float warp_total(uint64_t pair) {
  float lo, hi;
  f2_unpack(pair, lo, hi);
  lo += hi;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lo += __shfl_xor_sync(0xffffffffu, lo, o);
  return lo;
}

// Warps of a CTA: as many as the registers of a row (and of its passes) leave room for.
constexpr int row_warps(int nch) { return nch <= 4 ? 24 : nch <= 8 ? 20 : nch <= 12 ? 16 : 12; }

template <int NCH>
__global__ void __launch_bounds__(row_warps(NCH) * 32, 1)
    layer_norm_rows_kernel(const mf_bf16* __restrict__ x, const float* __restrict__ gamma,
                           const float* __restrict__ beta, const LnArgs a, float eps,
                           mf_bf16* __restrict__ y, float2* __restrict__ stats) {
  extern __shared__ float4 par[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nc = a.hid >> 3;
  const float inv_n = 1.f / static_cast<float>(a.hid);
  constexpr int kRowWarps = row_warps(NCH);
  const int row0 = blockIdx.x * kRowWarps + warp, stride = gridDim.x * kRowWarps;
  uint4 v[NCH];
  pdl_wait();
  pdl_release();
  for (int i = threadIdx.x; i < 8 * nc; i += blockDim.x) {
    // i: ((modality * 2 + which) * 2 + half) * nc + chunk
    const int chunk = i % nc, r = i / nc;
    const float* src = (r & 2) ? beta : gamma;
    par[i] = __ldg(reinterpret_cast<const float4*>(src + static_cast<size_t>(r >> 2) * a.hid) +
                   2 * chunk + (r & 1));
  }
  __syncthreads();
  for (int row = row0; row < a.T; row += stride) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + static_cast<size_t>(row) * a.hid);
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      const int i = lane + 32 * u;
      v[u] = i < nc ? __ldcs(xr + i) : make_uint4(0, 0, 0, 0);
    }
    const int m = __ldg(a.tok_mod + row);
    uint64_t acc = 0;
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      uint64_t f[4];
      bf16x8_f2(v[u], f);
      acc = f2_add(acc, f2_add(f2_add(f[0], f[1]), f2_add(f[2], f[3])));
    }
    const float mean = warp_total(acc) * inv_n;
    const uint64_t shift = f2_both(-mean);
    acc = 0;
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      if (lane + 32 * u < nc) {
        uint64_t f[4];
        bf16x8_f2(v[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t d = f2_add(f[e], shift);
          acc = f2_fma(d, d, acc);
        }
      }
    }
    const float rstd = rsqrtf(fmaf(warp_total(acc), inv_n, eps));
    if (m > 1) {
      if (lane == 0) atomicCAS(a.ctl.err, 0, static_cast<int>(MF_ERR_INVALID));
      continue;
    }
    const uint64_t scale = f2_both(rstd);
    const ulonglong2* p = reinterpret_cast<const ulonglong2*>(par + m * 4 * nc);
    uint4* yr = reinterpret_cast<uint4*>(y + static_cast<size_t>(row) * a.hid);
#pragma unroll
    for (int u = 0; u < NCH; ++u) {
      const int i = lane + 32 * u;
      if (i < nc) {
        uint64_t f[4];
        bf16x8_f2(v[u], f);
        const ulonglong2 g0 = p[i], g1 = p[nc + i], b0 = p[2 * nc + i], b1 = p[3 * nc + i];
        f[0] = f2_fma(f2_mul(f2_add(f[0], shift), scale), g0.x, b0.x);
        f[1] = f2_fma(f2_mul(f2_add(f[1], shift), scale), g0.y, b0.y);
        f[2] = f2_fma(f2_mul(f2_add(f[2], shift), scale), g1.x, b1.x);
        f[3] = f2_fma(f2_mul(f2_add(f[3], shift), scale), g1.y, b1.y);
        __stcs(yr + i, f2_bf16x8(f));
      }
    }
    if (lane == 0 && stats != nullptr) stats[row] = make_float2(mean, rstd);
  }
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bytes of one stage's parts (x, dy, resid), each a multiple of 128.
struct BwdStage {
  int x, d, r, stages;
  __host__ __device__ int bytes() const { return x + d + r; }
};

constexpr int kBwdRows = 2;  // rows per group and step: an even number, so that a
                             // step's 8-bit codes start on a 16-byte boundary
constexpr int kMaxStages = 4;

// A thread owns CH chunks of eight channels, a.lanes chunks apart; FULL: all of them
// exist (hid is 8 CH lanes), so nothing is guarded by the width. Dynamic shared
// memory: the stages, then, with more than one group, the groups' places for sums of
// a modality that ended, [groups][2 modalities][2 (dgamma, dbeta)][hid] fp32. A
// single group's place is part[blockIdx.x][2][2][hid] in memory, and at the end its
// totals stand in the stages' memory. sums_out[cluster][2][2][hid] (dgamma and dbeta
// themselves where there is one cluster, sums_out NULL) gets the cluster's sums; a
// cluster of several CTAs has one group in each.
template <int SUB, int CH, int THREADS, int PER_SM, bool FULL, bool X8>
__global__ void __launch_bounds__(THREADS, PER_SM) layer_norm_bwd_kernel(
    const mf_bf16* __restrict__ dy, const mf_bf16* __restrict__ x, const Act8 x8,
    const float* __restrict__ gamma, const float2* __restrict__ stats, const mf_bf16* resid,
    const LnArgs a, const BwdStage sg, mf_bf16* dx, float* __restrict__ part,
    float* __restrict__ sums_out, int cluster, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  constexpr int R = kBwdRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][32][2 * R];
  __shared__ uint64_t full[kMaxStages];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int group = threadIdx.x / a.lanes, gl = threadIdx.x - group * a.lanes;
  const int warps = a.lanes / 32, lane = threadIdx.x & 31;
  bool on[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) on[j] = FULL || (gl + j * a.lanes) * 8 < a.hid;
  const float inv_n = 1.f / static_cast<float>(a.hid);
  const int nb = (a.hid + kAct8Block - 1) / kAct8Block;
  int r0, r1;
  cta_rows<R>(a, r0, r1);
  const int step = a.groups * R;
  const int steps = (r1 - r0 + step - 1) / step;
  const int stage_bytes = sg.bytes();
  float* cols = reinterpret_cast<float*>(smem + sg.stages * stage_bytes);

  if (threadIdx.x == 0) {
    for (int i = 0; i < sg.stages; ++i) mbar_init(&full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_release();
  // thread 0: the rows of step s into stage `at`
  auto issue = [&](int s, int at) {
    const int row = r0 + s * step, rows = min(step, r1 - row);
    uint8_t* dst = smem + at * stage_bytes;
    uint64_t* bar = &full[at];
    const size_t off = static_cast<size_t>(row) * a.hid;
    const uint32_t n = static_cast<uint32_t>(rows) * a.hid;
    uint32_t nx = 2 * n;
    if constexpr (X8) {
      nx = n & ~15u;
      if (n & 8u)  // an odd last row of an odd width: its last eight codes
        *reinterpret_cast<uint2*>(dst + nx) = *reinterpret_cast<const uint2*>(x8.q + off + nx);
    }
    mbar_expect_tx(bar, nx + 2 * n + (resid != nullptr ? 2 * n : 0));
    if (nx > 0) {
      if constexpr (X8)
        bulk_load(dst, x8.q + off, nx, bar);
      else
        bulk_load(dst, x + off, nx, bar);
    }
    bulk_load(dst + sg.x, dy + off, 2 * n, bar);
    if (resid != nullptr) bulk_load(dst + sg.x + sg.d, resid + off, 2 * n, bar);
  };
  int issued = 0;  // thread 0: steps whose copies it has started
  if (threadIdx.x == 0)
    for (; issued < sg.stages && issued < steps; ++issued) issue(issued, issued);

  uint64_t gam[CH][4], ag[CH][4], ab[CH][4];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) gam[j][e] = ag[j][e] = ab[j][e] = 0;
  int cm = -1, seen = 0;
  // this group's place for modality m: dgamma's row, dbeta's row
  auto place = [&](int m, float*& g, float*& b) {
    g = (a.groups > 1 ? cols + static_cast<size_t>(group) * 4 * a.hid
                      : part + static_cast<size_t>(blockIdx.x) * 4 * a.hid) + m * 2 * a.hid;
    b = g + a.hid;
  };
  auto flush = [&]() {
    if (cm < 0) return;
    float *g, *b;
    place(cm, g, b);
    const bool more = (seen >> cm) & 1;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!on[j]) continue;
      uint64_t* g2 = reinterpret_cast<uint64_t*>(g + (gl + j * a.lanes) * 8);
      uint64_t* b2 = reinterpret_cast<uint64_t*>(b + (gl + j * a.lanes) * 8);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g2[e] = more ? f2_add(g2[e], ag[j][e]) : ag[j][e];
        b2[e] = more ? f2_add(b2[e], ab[j][e]) : ab[j][e];
        ag[j][e] = ab[j][e] = 0;
      }
    }
    seen |= 1 << cm;
  };
  // small per-row values of a step, fetched one step ahead
  float2 nst[R];
  float nsc[R][CH];
  int nmod[R];
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      nmod[i] = -1;
      nst[i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < CH; ++j) nsc[i][j] = 0.f;
      if (row + i < r1) {
        nmod[i] = __ldg(a.tok_mod + row + i);
        nst[i] = __ldg(stats + row + i);
        if constexpr (X8) {
          const float* sc = x8.scale + static_cast<size_t>(row + i) * nb;
#pragma unroll
          for (int j = 0; j < CH; ++j)
            if (on[j]) nsc[i][j] = __ldg(sc + (gl + j * a.lanes) * 8 / kAct8Block);
        }
      }
    }
  };
  int row = r0 + group * R;
  const uint32_t elem = static_cast<uint32_t>(group * R) * a.hid + gl * 8;  // within a stage
  const uint32_t chunk = a.lanes * 8;
  mf_bf16* out = dx + static_cast<size_t>(row) * a.hid + gl * 8;
  const size_t out_step = static_cast<size_t>(step) * a.hid;
  int at = 0, prev = 0;
  uint32_t parity = 0;
  fetch(row);
  for (int s = 0; s < steps; ++s, row += step, out += out_step) {
    float2 st[R];  // (-mean, rstd)
    float sc[R][CH];
    int mod[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      st[i] = make_float2(-nst[i].x, nst[i].y);
#pragma unroll
      for (int j = 0; j < CH; ++j) sc[i][j] = nsc[i][j];
      mod[i] = nmod[i];
      if (mod[i] > 1) {
        if (gl == 0) atomicCAS(a.ctl.err, 0, static_cast<int>(MF_ERR_INVALID));
        mod[i] = -1;
      }
    }
    fetch(row + step);
    const uint8_t* sx = smem + at * stage_bytes;
    const uint8_t* sd = sx + sg.x + 2 * elem;
    const uint8_t* sr = sd + sg.d;
    sx += X8 ? elem : 2 * elem;
    // A wait that runs out is recorded and the step goes on, so that every thread
    // still meets every barrier; no copy is started after it.
    (void)mbar_wait(&full[at], parity, a.ctl, abort_flag);
    auto operands = [&](int i, int j, uint64_t (&h)[4], uint64_t (&d)[4]) {
      const uint32_t o = i * a.hid + j * chunk;
      // (x - mean) rstd, the difference first: x rstd - mean rstd would leave the rounding of
      // a product where x is near the mean (one instruction a pair less: 65.4 against
      // 66.7 us at 16384 x 3072 from bf16, no difference with a residual or from 8 bits)
      const uint64_t r2 = f2_both(st[i].y), m2 = f2_both(st[i].x);
      if constexpr (X8) {
        act8_codes(*reinterpret_cast<const uint2*>(sx + o), h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = f2_fma(h[e], f2_both(sc[i][j]), m2);
      } else {
        bf16x8_f2(*reinterpret_cast<const uint4*>(sx + 2 * o), h);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = f2_add(h[e], m2);
      }
      bf16x8_f2(*reinterpret_cast<const uint4*>(sd + 2 * o), d);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = f2_mul(h[e], r2);
    };
    float sums[2 * R];
    auto accumulate = [&](int i) {
      uint64_t s1 = 0, s2 = 0;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!on[j]) continue;
        uint64_t h[4], d[4];
        operands(i, j, h, d);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ag[j][e] = f2_fma(d[e], h[e], ag[j][e]);
          ab[j][e] = f2_add(ab[j][e], d[e]);
          const uint64_t g = f2_mul(d[e], gam[j][e]);
          s1 = f2_add(s1, g);
          s2 = f2_fma(g, h[e], s2);
        }
      }
      float lo, hi;
      f2_unpack(s1, lo, hi);
      sums[2 * i] = lo + hi;
      f2_unpack(s2, lo, hi);
      sums[2 * i + 1] = lo + hi;
    };
    // nearly every step is of one modality throughout: one test, no more
    bool usual = cm >= 0;
#pragma unroll
    for (int i = 0; i < R; ++i) usual = usual && mod[i] == cm;
    if (usual) {
#pragma unroll
      for (int i = 0; i < R; ++i) accumulate(i);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        sums[2 * i] = sums[2 * i + 1] = 0.f;
        if (mod[i] < 0) continue;
        if (mod[i] != cm) {
          flush();
          cm = mod[i];
#pragma unroll
          for (int j = 0; j < CH; ++j)
            if (on[j])
              load8_f2(gamma + static_cast<size_t>(cm) * a.hid + (gl + j * a.lanes) * 8, gam[j]);
        }
        accumulate(i);
      }
    }
    // The four sums over a group's lanes. Lane l ends with sum l mod 4: two rounds
    // that halve the sums a lane holds, then plain ones (6 shuffles in place of 20).
    float part4;
    {
      const bool odd = lane & 1, upper = lane & 2;
      float k0 = odd ? sums[1] : sums[0], g0 = odd ? sums[0] : sums[1];
      float k1 = odd ? sums[3] : sums[2], g1 = odd ? sums[2] : sums[3];
      k0 += __shfl_xor_sync(0xffffffffu, g0, 1);
      k1 += __shfl_xor_sync(0xffffffffu, g1, 1);
      part4 = upper ? k1 : k0;
      part4 += __shfl_xor_sync(0xffffffffu, upper ? k0 : k1, 2);
    }
#pragma unroll
    for (int o = 4; o < SUB; o <<= 1) part4 += __shfl_xor_sync(0xffffffffu, part4, o);
    if (SUB == 32 && warps > 1 && lane < 4) red[s & 1][threadIdx.x >> 5][lane] = part4;
    __syncthreads();
    // every thread has left the previous step, so its stage can be filled again
    if (threadIdx.x == 0 && s > 0 && issued < steps && !*abort_flag) issue(issued++, prev);
    if (SUB == 32 && warps > 1) {
      // sum l mod 4 of the group's warps, eight of them at a time
      part4 = 0.f;
      for (int w = lane >> 2; w < warps; w += 8) part4 += red[s & 1][group * warps + w][lane & 3];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) part4 += __shfl_xor_sync(0xffffffffu, part4, o);
    }
    part4 *= -inv_n;
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) sums[i] = __shfl_sync(0xffffffffu, part4, (lane & ~3) | i);
    // `other`: a row before the step's change of modality, its weights read again
    auto finish = [&](int i, bool other) {
      const uint64_t m1 = f2_both(sums[2 * i]), m2 = f2_both(sums[2 * i + 1]);
      const uint64_t r2 = f2_both(st[i].y);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!on[j]) continue;
        uint64_t h[4], d[4], w[4], o[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = gam[j][e];
        if (other)
          load8_f2(gamma + static_cast<size_t>(mod[i]) * a.hid + (gl + j * a.lanes) * 8, w);
        operands(i, j, h, d);
        if (resid != nullptr)
          bf16x8_f2(*reinterpret_cast<const uint4*>(sr + 2 * (i * a.hid + j * chunk)), o);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = f2_fma(f2_fma(h[e], m2, f2_fma(d[e], w[e], m1)), r2, o[e]);
        *reinterpret_cast<uint4*>(out + static_cast<size_t>(i) * a.hid + j * chunk) = f2_bf16x8(o);
      }
    };
    if (usual) {
#pragma unroll
      for (int i = 0; i < R; ++i) finish(i, false);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (mod[i] >= 0) finish(i, mod[i] != cm);
    }
    prev = at;
    if (++at == sg.stages) {
      at = 0;
      parity ^= 1;
    }
  }
  // After a wait that ran out the last copies may still be under way; otherwise every
  // one has been waited for.
  if (threadIdx.x == 0 && *abort_flag)
    for (int s = max(0, issued - sg.stages); s < issued; ++s)
      drain_wait(&full[s % sg.stages], (s / sg.stages) & 1, a.ctl.wait_limit_ns);
  // The group's totals: what it put aside, and what it still holds.
  __syncthreads();  // the stages are free
  float* total = reinterpret_cast<float*>(smem);  // of a single group
  float* mine = a.groups > 1 ? cols + static_cast<size_t>(group) * 4 * a.hid : total;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float *g, *b;
    place(m, g, b);
    const bool more = (seen >> m) & 1, held = m == cm;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!on[j]) continue;
      const int c = (gl + j * a.lanes) * 8;
      const uint64_t* g2 = reinterpret_cast<const uint64_t*>(g + c);
      const uint64_t* b2 = reinterpret_cast<const uint64_t*>(b + c);
      uint64_t* to_g = reinterpret_cast<uint64_t*>(mine + 2 * m * a.hid + c);
      uint64_t* to_b = reinterpret_cast<uint64_t*>(mine + (2 * m + 1) * a.hid + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint64_t vg = held ? ag[j][e] : 0, vb = held ? ab[j][e] : 0;
        if (more) {
          vg = f2_add(g2[e], vg);
          vb = f2_add(b2[e], vb);
        }
        to_g[e] = vg;
        to_b[e] = vb;
      }
    }
  }
  // The CTA's groups in order, or the cluster's CTAs (a cluster's have one group each),
  // four columns at a time; each CTA of a cluster adds every cluster-th four.
  if (cluster > 1) cluster_sync();
  else __syncthreads();
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const float* first = a.groups > 1 ? cols : total;
  for (int i = (threadIdx.x * cluster + rank) * 4; i < 4 * a.hid; i += blockDim.x * cluster * 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < (cluster > 1 ? cluster : a.groups); ++q) {
      float4 w;
      if (cluster > 1)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                     : "r"(cluster_addr(first + i, q))
                     : "memory");
      else
        w = *reinterpret_cast<const float4*>(first + static_cast<size_t>(q) * 4 * a.hid + i);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    float* to;
    if (sums_out != nullptr) {
      to = sums_out + static_cast<size_t>(blockIdx.x / cluster) * 4 * a.hid + i;
    } else {
      const int m = i / (2 * a.hid), r = i - m * 2 * a.hid;
      to = (r < a.hid ? dgamma : dbeta) + m * a.hid + (r < a.hid ? r : r - a.hid);
    }
    *reinterpret_cast<float4*>(to) = v;
  }
  if (cluster > 1) cluster_sync();  // no CTA leaves while another reads its totals
}

// dgamma / dbeta = the sum over the n partials, in a fixed order: 32 columns per
// CTA, 32 slices of the partials, one warp each, then the slices in order.
__global__ void __launch_bounds__(1024) ln_cols_kernel(const float* __restrict__ part, int n,
                                                       int hid, float* __restrict__ dgamma,
                                                       float* __restrict__ dbeta) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  pdl_wait();
  pdl_release();
  float v = 0.f;
  if (col < 4 * hid) {
#pragma unroll 10
    for (int k = slice; k < n; k += 32) v += __ldcg(part + static_cast<size_t>(k) * 4 * hid + col);
  }
  s[slice][lane] = v;
  __syncthreads();
  // warp w: columns w, 32 slices by shuffles
  v = s[lane][slice];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int c = blockIdx.x * 32 + slice;
  if (lane == 0 && c < 4 * hid) {
    const int m = c / (2 * hid), r = c - m * 2 * hid;
    (r < hid ? dgamma : dbeta)[m * hid + (r < hid ? r : r - hid)] = v;
  }
}

template <int SUB, int R, int THREADS>
cudaError_t fwd_shape(const mf_bf16* x, const float* gamma, const float* beta, const LnArgs& a,
                      int threads, float eps, mf_bf16* y, float* stats, cudaStream_t st) {
  const int steps = (a.T + a.groups * R - 1) / (a.groups * R);
  const int cap = ln_sms() * (threads > 512 ? 1 : threads > 256 ? 2 : 4);
  return launch_dependent(layer_norm_kernel<SUB, R, THREADS>, dim3(steps < cap ? steps : cap),
                          dim3(threads), 0, st, x, gamma, beta, a, eps, y,
                          reinterpret_cast<float2*>(stats));
}

template <int NCH>
cudaError_t fwd_rows(const mf_bf16* x, const float* gamma, const float* beta, const LnArgs& a,
                     float eps, mf_bf16* y, float* stats, cudaStream_t st) {
  auto kernel = layer_norm_rows_kernel<NCH>;
  // the limit of every width the instance takes: calls of two threads do not lower
  // each other's
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NCH * 256 * 16);
  if (e != cudaSuccess) return e;
  const int smem = a.hid * 16;
  constexpr int kRowWarps = row_warps(NCH);
  const int need = (a.T + kRowWarps - 1) / kRowWarps, cap = ln_sms();
  return launch_dependent(kernel, dim3(need < cap ? need : cap), dim3(kRowWarps * 32), smem, st, x,
                          gamma, beta, a, eps, y, reinterpret_cast<float2*>(stats));
}

// How the backward shares rows: as the forward up to 2048 channels, then two chunks
// per thread, which halves what a row costs beside its values.
RowShape bwd_row_shape(int32_t hid) {
  if (hid <= 2048) return row_shape(hid);
  RowShape s;
  s.lanes = (hid / 8 + 63) / 64 * 32;
  s.groups = 1;
  s.threads = s.lanes;
  return s;
}

// CTAs per SM: several, so that one computes while another waits at its barrier; one
// above 256 threads, whose registers leave no more room.
int bwd_per_sm(const RowShape& s) { return s.threads > 256 ? 1 : 2; }

constexpr int kBwdSmem = 222 * 1024;  // an SM's shared memory, the kernel's own 1 KB aside

BwdStage bwd_stage(const RowShape& s, int32_t hid, bool x8, bool resid) {
  auto round128 = [](int v) { return (v + 127) / 128 * 128; };
  const int n = s.groups * kBwdRows * hid;
  BwdStage g;
  g.x = round128(x8 ? n : 2 * n);
  g.d = round128(2 * n);
  g.r = resid ? g.d : 0;
  const int cols = s.groups > 1 ? s.groups * 16 * hid : 0;
  const int room = kBwdSmem / bwd_per_sm(s) - 2048 - cols;
  g.stages = room / g.bytes();
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  return g;
}

// One CTA per step up to one per SM, then one per four steps: each CTA leaves column
// sums for the second kernel to add.
int bwd_grid(const RowShape& s, int32_t T) {
  const int steps = (T + s.groups * kBwdRows - 1) / (s.groups * kBwdRows), sms = ln_sms();
  if (steps <= sms) return steps;
  const int by_steps = steps / 4, cap = sms * bwd_per_sm(s);
  return (by_steps < sms ? sms : by_steps < cap ? by_steps : cap) / 2 * 2;
}

// CTAs that add their sums before they leave: pairs in wide rows, where that halves
// what the second kernel reads (84 -> 78 us at 16384 x 3072, 38.2 -> 34.6 at 8464 x
// 2048; 18.6 -> 19.8 at 4837 x 1000). Pairs all fit at once; clusters of four leave
// SMs of a GPC out and come in two waves (117 us at 16384 x 3072).
// Above 1024 channels a CTA has one group.
int bwd_cluster(int grid, int32_t hid) { return hid > 1024 && grid % 2 == 0 ? 2 : 1; }

template <int SUB, int CH, int THREADS, int PER_SM, bool FULL, bool X8>
cudaError_t bwd_shape(const mf_bf16* dy, const mf_bf16* x, const Act8& x8, const float* gamma,
                      const float* stats, const mf_bf16* resid, const LnArgs& a, const RowShape& s,
                      mf_bf16* dx, float* dgamma, float* dbeta, float* part, cudaStream_t st) {
  auto kernel = layer_norm_bwd_kernel<SUB, CH, THREADS, PER_SM, FULL, X8>;
  const BwdStage g = bwd_stage(s, a.hid, X8, resid != nullptr);
  const int smem = g.stages * g.bytes() + (s.groups > 1 ? s.groups * 16 * a.hid : 0);
  const cudaError_t ae =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
  if (ae != cudaSuccess) return ae;
  const int grid = bwd_grid(s, a.T), cluster = bwd_cluster(grid, a.hid);
  const int clusters = grid / cluster;
  float* sums = clusters > 1 ? part + static_cast<size_t>(grid) * 4 * a.hid : nullptr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kernel, dy, x, x8, gamma, reinterpret_cast<const float2*>(stats),
                         resid, a, g, dx, part, sums, cluster, dgamma, dbeta);
  if (e != cudaSuccess || sums == nullptr) return e;
  return launch_dependent(ln_cols_kernel, dim3((4 * a.hid + 31) / 32), dim3(1024), 0, st, sums,
                          clusters, a.hid, dgamma, dbeta);
}

}  // namespace

cudaError_t launch_layer_norm(const mf_bf16* x, const float* gamma, const float* beta,
                              const uint8_t* tok_mod, int32_t T, int32_t hid, float eps,
                              mf_bf16* y, float* stats, const KernelCtl& ctl, cudaStream_t st) {
  const RowShape s = row_shape(hid);
  const LnArgs a{tok_mod, T, hid, s.lanes, s.groups, ctl};
  if (s.lanes == 8) return fwd_shape<8, 4, 256>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  if (s.lanes == 16) return fwd_shape<16, 4, 256>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  if (s.lanes == 32) return fwd_shape<32, 4, 256>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  if (hid <= 512) return fwd_rows<2>(x, gamma, beta, a, eps, y, stats, st);
  if (hid <= 1024) return fwd_rows<4>(x, gamma, beta, a, eps, y, stats, st);
  if (hid <= 2048) return fwd_rows<8>(x, gamma, beta, a, eps, y, stats, st);
  if (hid <= 3072) return fwd_rows<12>(x, gamma, beta, a, eps, y, stats, st);
  if (hid <= 4096) return fwd_rows<16>(x, gamma, beta, a, eps, y, stats, st);
  return fwd_shape<32, 2, 1024>(x, gamma, beta, a, s.threads, eps, y, stats, st);
}

size_t layer_norm_bwd_ws(int32_t T, int32_t hid) {
  return static_cast<size_t>(2 * bwd_grid(bwd_row_shape(hid), T)) * 4 * hid * sizeof(float);
}

cudaError_t launch_layer_norm_bwd(const mf_bf16* dy, const mf_bf16* x, const Act8& x8,
                                  const float* gamma, const float* stats, const uint8_t* tok_mod,
                                  const mf_bf16* resid, int32_t T, int32_t hid, mf_bf16* dx,
                                  float* dgamma, float* dbeta, void* ws, const KernelCtl& ctl,
                                  cudaStream_t st) {
  const RowShape s = bwd_row_shape(hid);
  const LnArgs a{tok_mod, T, hid, s.lanes, s.groups, ctl};
  float* part = reinterpret_cast<float*>(ws);
#define MF_LN_BWD(SUB, CH, THREADS, PER_SM, FULL)                                              \
  (x8.q != nullptr                                                                             \
       ? bwd_shape<SUB, CH, THREADS, PER_SM, FULL, true>(dy, x, x8, gamma, stats, resid, a, s, \
                                                         dx, dgamma, dbeta, part, st)          \
       : bwd_shape<SUB, CH, THREADS, PER_SM, FULL, false>(dy, x, x8, gamma, stats, resid, a, s, \
                                                          dx, dgamma, dbeta, part, st))
  if (s.lanes == 8) return MF_LN_BWD(8, 1, 256, 2, false);
  if (s.lanes == 16) return MF_LN_BWD(16, 1, 256, 2, false);
  if (hid <= 2048)
    return hid == 8 * s.lanes ? MF_LN_BWD(32, 1, 256, 2, true) : MF_LN_BWD(32, 1, 256, 2, false);
  const bool full = hid == 16 * s.lanes;
  if (hid <= 3072) return full ? MF_LN_BWD(32, 2, 192, 2, true) : MF_LN_BWD(32, 2, 192, 2, false);
  if (hid <= 4096) return full ? MF_LN_BWD(32, 2, 256, 2, true) : MF_LN_BWD(32, 2, 256, 2, false);
  return full ? MF_LN_BWD(32, 2, 512, 1, true) : MF_LN_BWD(32, 2, 512, 1, false);
#undef MF_LN_BWD
}

}  // namespace mf
