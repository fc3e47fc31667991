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
// writes dx. So that nothing else is read per row, a thread owns eight channels
// for the whole launch: their gamma, beta and, in the backward, their running
// dgamma and dbeta stay in registers, and a row is shared by a group of threads
// (8, 16 or 32 lanes, or several warps). A group takes R rows per step and has
// the next step's loads in flight while it reduces; the row sums are reduced by
// shuffles and, over several warps, through shared memory at one named barrier.
// The forward takes the variance about the mean in a second reduction over the
// rows in registers (no cancellation). The backward's column sums go, whenever
// the modality of a group's rows changes and at the end, to the group's own place
// in shared memory, then per CTA to the workspace, then through a second kernel
// that adds the CTAs in a fixed order: no atomics, the same bits every time.
#include <cuda_bf16.h>

#include <cstdint>

#include "act8.cuh"
#include "mlp_internal.h"

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

// part: [grid][2 modalities][2 (dgamma, dbeta)][hid], or dgamma / dbeta
// themselves when the grid is one CTA (part NULL). Shared memory:
// [groups][2][2][hid] fp32.
template <int SUB, int R, int THREADS, bool X8>
__global__ void __launch_bounds__(THREADS) layer_norm_bwd_kernel(
    const mf_bf16* __restrict__ dy, const mf_bf16* __restrict__ x, const Act8 x8,
    const float* __restrict__ gamma, const float2* __restrict__ stats, const mf_bf16* resid,
    const LnArgs a, mf_bf16* dx, float* __restrict__ part, float* __restrict__ dgamma,
    float* __restrict__ dbeta) {
  extern __shared__ float cols[];
  __shared__ float red[2 * 32 * 8];
  const int group = threadIdx.x / a.lanes, gl = threadIdx.x - group * a.lanes;
  const int warps = a.lanes / 32, wig = gl / 32;
  const int c = gl * 8;
  const bool on = c < a.hid;
  const float inv_n = 1.f / static_cast<float>(a.hid);
  const int nb = (a.hid + kAct8Block - 1) / kAct8Block;
  int r0, r1, flip = 0;
  cta_rows<R>(a, r0, r1);
  float* mine = cols + static_cast<size_t>(group) * 4 * a.hid;  // [2][2][hid]
  if (on) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) mine[j * a.hid + c + e] = 0.f;
  }
  float gam[8], ag[8], ab[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) gam[e] = ag[e] = ab[e] = 0.f;
  int cm = -1;
  auto flush = [&]() {
    if (on && cm >= 0) {
      float* p = mine + cm * 2 * a.hid + c;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] += ag[e];
        p[a.hid + e] += ab[e];
        ag[e] = ab[e] = 0.f;
      }
    }
  };
  uint4 nx[R], nd[R];
  float2 nst[R];
  float ns[R];
  int mod_next[R];
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool live = row + i < r1;
      mod_next[i] = live ? __ldg(a.tok_mod + row + i) : -1;
      nst[i] = live ? __ldg(stats + row + i) : make_float2(0.f, 0.f);
      const size_t off = static_cast<size_t>(row + i) * a.hid + c;
      nx[i] = nd[i] = make_uint4(0, 0, 0, 0);
      ns[i] = 0.f;
      if (live && on) {
        nd[i] = __ldcs(reinterpret_cast<const uint4*>(dy + off));
        if constexpr (X8) {
          const uint2 w = __ldcs(reinterpret_cast<const uint2*>(x8.q + off));
          nx[i].x = w.x;
          nx[i].y = w.y;
          ns[i] = __ldg(x8.scale + static_cast<size_t>(row + i) * nb + c / kAct8Block);
        } else {
          nx[i] = __ldcs(reinterpret_cast<const uint4*>(x + off));
        }
      }
    }
  };
  const int step = a.groups * R;
  fetch(r0 + group * R);
  // every group of the CTA takes the same number of steps: its rows past the end
  // are not live, but its lanes shuffle with their warp's other groups
  for (int base = r0; base < r1; base += step) {
    const int row = base + group * R;
    uint4 vx[R], vd[R], vr[R];
    float2 st[R];
    float sc[R];
    int mod[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      vx[i] = nx[i];
      vd[i] = nd[i];
      st[i] = nst[i];
      sc[i] = ns[i];
      mod[i] = mod_next[i];
      vr[i] = make_uint4(0, 0, 0, 0);
      if (resid != nullptr && on && row + i < r1)
        vr[i] = *reinterpret_cast<const uint4*>(resid + static_cast<size_t>(row + i) * a.hid + c);
    }
    fetch(row + step);
    auto xhat = [&](int i, float (&h)[8]) {
      if constexpr (X8)
        act8_load(make_uint2(vx[i].x, vx[i].y), sc[i], h);
      else
        bf16x8_unpack(vx[i], h);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = (h[e] - st[i].x) * st[i].y;
    };
    // the modality's weights, then the row sums of g and g xhat
    float sums[2 * R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      sums[2 * i] = sums[2 * i + 1] = 0.f;
      if (mod[i] < 0 || mod[i] > 1) {
        if (mod[i] > 1 && gl == 0) atomicCAS(a.ctl.err, 0, static_cast<int>(MF_ERR_INVALID));
        continue;
      }
      if (mod[i] != cm) {
        flush();
        cm = mod[i];
        if (on) load8(gamma + static_cast<size_t>(cm) * a.hid + c, gam);
      }
      float h[8], d[8];
      xhat(i, h);
      bf16x8_unpack(vd[i], d);
      if (on) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ag[e] = fmaf(d[e], h[e], ag[e]);
          ab[e] += d[e];
          const float g = d[e] * gam[e];
          sums[2 * i] += g;
          sums[2 * i + 1] = fmaf(g, h[e], sums[2 * i + 1]);
        }
      }
    }
    group_sum<2 * R, SUB>(sums, warps, group, wig, red, flip);
    float gm[8];
    int gmod = cm;
#pragma unroll
    for (int e = 0; e < 8; ++e) gm[e] = gam[e];
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      if (mod[i] < 0 || mod[i] > 1) continue;
      if (mod[i] != gmod) {  // an earlier row of the step, before the change
        gmod = mod[i];
        if (on) load8(gamma + static_cast<size_t>(gmod) * a.hid + c, gm);
      }
      if (!on) continue;
      float h[8], d[8], o[8];
      xhat(i, h);
      bf16x8_unpack(vd[i], d);
      bf16x8_unpack(vr[i], o);
      const float m1 = sums[2 * i] * inv_n, m2 = sums[2 * i + 1] * inv_n;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = fmaf(d[e] * gm[e] - m1 - h[e] * m2, st[i].y, o[e]);
      *reinterpret_cast<uint4*>(dx + static_cast<size_t>(row + i) * a.hid + c) = bf16x8_pack(o);
    }
  }
  flush();
  __syncthreads();
  // the CTA's groups in order
  for (int i = threadIdx.x; i < 4 * a.hid; i += blockDim.x) {
    float v = 0.f;
    for (int g = 0; g < a.groups; ++g) v += cols[static_cast<size_t>(g) * 4 * a.hid + i];
    if (part != nullptr) {
      part[static_cast<size_t>(blockIdx.x) * 4 * a.hid + i] = v;
    } else {
      const int m = i / (2 * a.hid), r = i - m * 2 * a.hid;
      (r < a.hid ? dgamma : dbeta)[m * a.hid + (r < a.hid ? r : r - a.hid)] = v;
    }
  }
}

// dgamma / dbeta = the sum over the n partials, in a fixed order: 32 columns per
// CTA, eight slices of the partials each, then the slices in order.
__global__ void __launch_bounds__(256) ln_cols_kernel(const float* __restrict__ part, int n,
                                                      int hid, float* __restrict__ dgamma,
                                                      float* __restrict__ dbeta) {
  __shared__ float s[8][32];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float v = 0.f;
  if (col < 4 * hid) {
#pragma unroll 8
    for (int k = slice; k < n; k += 8) v += __ldg(part + static_cast<size_t>(k) * 4 * hid + col);
  }
  s[slice][threadIdx.x & 31] = v;
  __syncthreads();
  if (slice == 0 && col < 4 * hid) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x & 31];
    const int m = col / (2 * hid), r = col - m * 2 * hid;
    (r < hid ? dgamma : dbeta)[m * hid + (r < hid ? r : r - hid)] = v;
  }
}

template <int SUB, int R, int THREADS>
cudaError_t fwd_shape(const mf_bf16* x, const float* gamma, const float* beta, const LnArgs& a,
                      int threads, float eps, mf_bf16* y, float* stats, cudaStream_t st) {
  const int steps = (a.T + a.groups * R - 1) / (a.groups * R);
  const int cap = ln_sms() * (threads > 512 ? 1 : threads > 256 ? 2 : 4);
  layer_norm_kernel<SUB, R, THREADS><<<steps < cap ? steps : cap, threads, 0, st>>>(
      x, gamma, beta, a, eps, y, reinterpret_cast<float2*>(stats));
  return cudaGetLastError();
}

int bwd_cap(int threads) { return ln_sms() * (threads > 256 ? 1 : 2); }

template <int SUB, int R, int THREADS, bool X8>
cudaError_t bwd_shape(const mf_bf16* dy, const mf_bf16* x, const Act8& x8, const float* gamma,
                      const float* stats, const mf_bf16* resid, const LnArgs& a, int threads,
                      mf_bf16* dx, float* dgamma, float* dbeta, float* part, cudaStream_t st) {
  auto kernel = layer_norm_bwd_kernel<SUB, R, THREADS, X8>;
  const size_t smem = static_cast<size_t>(a.groups) * 4 * a.hid * sizeof(float);
  if (smem > 40960) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const int steps = (a.T + a.groups * R - 1) / (a.groups * R);
  const int cap = bwd_cap(threads);
  const int grid = steps < cap ? steps : cap;
  float* p = grid > 1 ? part : nullptr;
  kernel<<<grid, threads, smem, st>>>(dy, x, x8, gamma, reinterpret_cast<const float2*>(stats),
                                      resid, a, dx, p, dgamma, dbeta);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p == nullptr) return e;
  ln_cols_kernel<<<(4 * a.hid + 31) / 32, 256, 0, st>>>(p, grid, a.hid, dgamma, dbeta);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_layer_norm(const mf_bf16* x, const float* gamma, const float* beta,
                              const uint8_t* tok_mod, int32_t T, int32_t hid, float eps,
                              mf_bf16* y, float* stats, const KernelCtl& ctl, cudaStream_t st) {
  const RowShape s = row_shape(hid);
  const LnArgs a{tok_mod, T, hid, s.lanes, s.groups, ctl};
  if (s.lanes == 8) return fwd_shape<8, 4, 256>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  if (s.lanes == 16) return fwd_shape<16, 4, 256>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  if (s.threads <= 512)
    return fwd_shape<32, 4, 512>(x, gamma, beta, a, s.threads, eps, y, stats, st);
  return fwd_shape<32, 2, 1024>(x, gamma, beta, a, s.threads, eps, y, stats, st);
}

size_t layer_norm_bwd_ws(int32_t T, int32_t hid) {
  (void)T;
  return static_cast<size_t>(bwd_cap(row_shape(hid).threads)) * 4 * hid * sizeof(float);
}

cudaError_t launch_layer_norm_bwd(const mf_bf16* dy, const mf_bf16* x, const Act8& x8,
                                  const float* gamma, const float* stats, const uint8_t* tok_mod,
                                  const mf_bf16* resid, int32_t T, int32_t hid, mf_bf16* dx,
                                  float* dgamma, float* dbeta, void* ws, const KernelCtl& ctl,
                                  cudaStream_t st) {
  const RowShape s = row_shape(hid);
  const LnArgs a{tok_mod, T, hid, s.lanes, s.groups, ctl};
  float* part = reinterpret_cast<float*>(ws);
#define MF_LN_BWD(SUB, R, THREADS)                                                               \
  (x8.q != nullptr ? bwd_shape<SUB, R, THREADS, true>(dy, x, x8, gamma, stats, resid, a,         \
                                                      s.threads, dx, dgamma, dbeta, part, st)    \
                   : bwd_shape<SUB, R, THREADS, false>(dy, x, x8, gamma, stats, resid, a,        \
                                                       s.threads, dx, dgamma, dbeta, part, st))
  if (s.lanes == 8) return MF_LN_BWD(8, 2, 256);
  if (s.lanes == 16) return MF_LN_BWD(16, 2, 256);
  if (s.threads <= 512) return MF_LN_BWD(32, 2, 512);
  return MF_LN_BWD(32, 1, 1024);
#undef MF_LN_BWD
}

}  // namespace mf
