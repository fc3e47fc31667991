// linear_rows.cu -- the fused linear layer and its input gradient for few rows (up to
// 128 tokens: a prompt, a single token): the products of linear_fused.cu with the
// roles of the operands exchanged.
//
// With few rows the time is that of reading the weights once. A 256-row tile would
// leave most of a tensor-core tile empty and, at 256 output columns a tile, most SMs
// without work. So 128 outputs (rows of W, or columns of it for dx) are the M of the
// MMAs and the tokens, padded to 16, 32, 64 or 128, their N, and the inner dimension
// is cut over a cluster of up to eight CTAs, so that about two CTAs per SM stream
// weights (16 KB a step, 64 of the inner dimension). Each CTA leaves its part of the
// 128 x tokens tile in its shared memory; then every CTA takes its share of the
// tokens, adds the parts over the cluster in order (distributed shared memory; no
// atomics, the same bits every time) and runs the epilogue: a token's 128 outputs lie
// in one warp, four to a lane, which is also one block of an 8-bit checkpoint.
// Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "act8.cuh"
#include "linear_common.cuh"
#include "mf_internal.h"
#include "mf_ptx.cuh"
#include "mlp_internal.h"
#include "pdl.cuh"

namespace mf {

namespace {

constexpr int kOut = 128;    // outputs of a tile (MMA M)
constexpr int kStepK = 64;   // inner dimension per step: one 128-byte swizzle atom
constexpr int kWBytes = kOut * kStepK * 2;
constexpr int kBoxBytes = 64 * 64 * 2;
constexpr int kThreads = 128;
constexpr int kMaxStages = 6;
constexpr int kPartPad = 4;  // floats behind a token's 128, against bank conflicts
constexpr int kSmemBudget = 112 * 1024;  // two CTAs per SM

struct RowsArgs {
  int32_t T, outs, inner;  // tokens, outputs, inner dimension
  int32_t tiles, steps, splits;
  int32_t nt;              // tokens, padded
  int32_t stages, tmem_cols;
  int32_t job_m[2];        // modality of each job (gridDim / (splits * tiles) of them)
  const uint8_t* tok_mod;
  LinearEpilogue ep;       // dx: only out
  KernelCtl ctl;
};

__device__ __forceinline__ void load_3d_by(bool leader, void* dst, const CUtensorMap* map,
                                           uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

__device__ __forceinline__ float4 load_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Four outputs of a token, rounded to bf16.
__device__ __forceinline__ uint2 pack4(const float (&f)[4]) {
  return make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
}

template <int ACT>
__device__ __forceinline__ void act4(float (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) f2_unpack(act_fwd2<ACT>(f2_pack(f[e], f[e + 1])), f[e], f[e + 1]);
}

// W_MN: dx, whose outputs run along W's contiguous dimension.
template <bool W_MN>
__global__ void __launch_bounds__(kThreads) linear_rows_kernel(
    const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
    const __grid_constant__ RowsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const int warp = warp_uniform(static_cast<int>(threadIdx.x) >> 5), lane = threadIdx.x & 31;
  const int stage_bytes = kWBytes + a.nt * kStepK * 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_w);
    tma_prefetch_map(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = warp_uniform(tmem_slot);
  pdl_wait();
  pdl_release();

  const int rank = warp_uniform(static_cast<int>(cluster_ctarank()));
  const int unit = static_cast<int>(blockIdx.x) / a.splits;
  const int job = unit / a.tiles, out0 = (unit - job * a.tiles) * kOut;
  const int m = a.job_m[job];
  const int s0 = a.steps * rank / a.splits, s1 = a.steps * (rank + 1) / a.splits;

  // Both loops below are run by all lanes and issued from by lane 0, so that addresses
  // and descriptors are in uniform registers.
  const bool leader = lane == 0;
  if (warp == 0) {
    int st = 0;
    uint32_t phase = 1;
    int issued = 0;
    for (int s = s0; s < s1; ++s, ++issued) {
      if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], phase, a.ctl, abort_flag))) break;
      uint8_t* sw = smem + st * stage_bytes;
      expect_by(leader, &full[st], stage_bytes);
      if constexpr (W_MN) {
        load_3d_by(leader, sw, &map_w, &full[st], out0, s * kStepK, m);
        load_3d_by(leader, sw + kBoxBytes, &map_w, &full[st], out0 + 64, s * kStepK, m);
      } else {
        load_3d_by(leader, sw, &map_w, &full[st], s * kStepK, out0, m);
      }
      load_2d_by(leader, sw + kWBytes, &map_x, &full[st], s * kStepK, 0);
      if (++st == a.stages) {
        st = 0;
        phase ^= 1;
      }
    }
    // every copy lands before the stages are used again below
    for (int i = 0; i < a.stages; ++i)
      if (issued > i)
        drain_wait(&full[i], ((issued - 1 - i) / a.stages) & 1, a.ctl.wait_limit_ns);
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16_f32(kOut, a.nt, W_MN, 0);
    constexpr uint64_t W_STEP = W_MN ? 128 : 2;
    const uint32_t base = warp_uniform(smem_u32(smem));
    int st = 0;
    uint32_t phase = 0;
    for (int s = s0; s < s1; ++s) {
      if (!__all_sync(0xffffffffu, mbar_wait(&full[st], phase, a.ctl, abort_flag))) break;
      tc_fence_after();
      const uint32_t at = base + st * stage_bytes;
      const uint64_t dw = sdesc_sw128(at, W_MN ? kBoxBytes : 16, 1024);
      const uint64_t dx = sdesc_sw128(at + kWBytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < kStepK / 16; ++kk)
        umma_ss_by(leader, tmem, dw + kk * W_STEP, dx + kk * 2, idesc, (s > s0 || kk > 0) ? 1u : 0u);
      umma_commit_by(leader, &empty[st]);
      if (++st == a.stages) {
        st = 0;
        phase ^= 1;
      }
    }
    umma_commit_by(leader, &done);
  }
  __syncwarp();
  // A wait that ran out is recorded; the CTA still meets its cluster at the barriers.
  (void)mbar_wait(&done, 0, a.ctl, abort_flag);
  __syncthreads();  // the producer has seen its last copies land, too
  tc_fence_after();

  // This CTA's part: part[token][output], a TMEM lane (an output) per thread.
  float* part = reinterpret_cast<float*>(smem);
  constexpr int kPitch = kOut + kPartPad;
  for (int c = 0; c < a.nt; c += 16) {
    uint32_t v[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
          "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c));
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      asm volatile("" : "+r"(v[e]));
      part[(c + e) * kPitch + threadIdx.x] = __uint_as_float(v[e]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }
  cluster_sync();

  // Token t belongs to CTA t mod splits; a warp takes one at a time.
  const int o = out0 + lane * 4;
  const bool on = o < a.outs;
  const LinearEpilogue& ep = a.ep;
  for (int t = warp * a.splits + rank; t < a.T; t += 4 * a.splits) {
    if (__ldg(a.tok_mod + t) != m) continue;
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const float* mine = part + t * kPitch + lane * 4;
    for (int q = 0; q < a.splits; ++q) {
      const float4 v = load_cluster(cluster_addr(mine, q));
      f[0] += v.x;
      f[1] += v.y;
      f[2] += v.z;
      f[3] += v.w;
    }
    const size_t off = static_cast<size_t>(t) * a.outs + o;
    if constexpr (!W_MN) {
      if (ep.bias != nullptr && on) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(ep.bias + static_cast<size_t>(m) * a.outs + o));
        f[0] += b.x;
        f[1] += b.y;
        f[2] += b.z;
        f[3] += b.w;
      }
      if (ep.z8 != nullptr) {
        uint32_t top = 0;
        if (on)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        float s, inv;
        act8_scale(__uint_as_float(top), s, inv);
        if (on)
          *reinterpret_cast<uint32_t*>(ep.z8 + off) =
              act8_code4(f2_pack(f[0], f[1]), f2_pack(f[2], f[3]), inv, inv == 0.f ? 0u : 0xFFFFFFFFu);
        if (lane == 0) ep.z_scale[static_cast<size_t>(t) * ((a.outs + kAct8Block - 1) / kAct8Block) + out0 / kAct8Block] = s;
      }
      if (ep.z != nullptr && on) *reinterpret_cast<uint2*>(ep.z + off) = pack4(f);
      if (ep.act == MF_ACT_GELU) act4<MF_ACT_GELU>(f);
      if (ep.act == MF_ACT_SILU) act4<MF_ACT_SILU>(f);
      if (ep.resid != nullptr && on) {
        const uint2 r = *reinterpret_cast<const uint2*>(ep.resid + off);
        f[0] += __uint_as_float(r.x << 16);
        f[1] += __uint_as_float(r.x & 0xFFFF0000u);
        f[2] += __uint_as_float(r.y << 16);
        f[3] += __uint_as_float(r.y & 0xFFFF0000u);
      }
    }
    if (on) *reinterpret_cast<uint2*>(ep.out + off) = pack4(f);
  }
  cluster_sync();  // no CTA leaves while another reads its part
}

int sm_count() {
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

template <bool W_MN>
bool ready() {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(linear_rows_kernel<W_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBudget) != cudaSuccess)
      return false;
    done[dev] = true;
  }
  return true;
}

// b [T][inner] (x, or dz), W [2][N][K], `outs` outputs per token.
template <bool W_MN>
cudaError_t launch_rows(const mf_bf16* b, const mf_bf16* W, const TokenRuns& runs,
                        const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                        const LinearEpilogue& ep, const KernelCtl& ctl, cudaStream_t st) {
  RowsArgs a;
  a.T = T;
  a.outs = W_MN ? K : N;
  a.inner = W_MN ? N : K;
  a.tiles = (a.outs + kOut - 1) / kOut;
  a.steps = (a.inner + kStepK - 1) / kStepK;
  a.nt = 16;
  while (a.nt < T) a.nt *= 2;
  a.tmem_cols = a.nt < 32 ? 32 : a.nt;
  const int stage = kWBytes + a.nt * kStepK * 2;
  a.stages = (kSmemBudget - 1024) / stage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  int jobs = 0;
  for (int m = 0; m < 2; ++m)
    if (runs.count[m] > 0) a.job_m[jobs++] = m;
  // The largest cluster of 1, 2, 4 or 8 with at most two CTAs per SM and four steps a
  // CTA at least. (Clusters of three, 288 CTAs for 96 tiles, do not all fit at once:
  // 26.2 us against 18.5 for 192 CTAs in clusters of two, 16 tokens, 3072 -> 12288.)
  const int units = a.tiles * jobs;
  a.splits = 1;
  while (a.splits < 8 && units * a.splits * 2 <= 2 * sm_count() && a.steps >= a.splits * 8)
    a.splits *= 2;
  a.tok_mod = tok_mod;
  a.ep = ep;
  a.ctl = ctl;
  CUtensorMap mw, mx;
  if (!linear_map(&mw, W, K, N, 2, W_MN ? kStepK : kOut) ||
      !linear_map(&mx, b, a.inner, T, 0, a.nt))
    return cudaErrorInvalidValue;
  if (!ready<W_MN>()) return cudaErrorInvalidConfiguration;
  // the parts use the stages' memory afterwards
  const int part = a.nt * (kOut + kPartPad) * static_cast<int>(sizeof(float));
  const int ring = a.stages * stage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units) * a.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (part > ring ? part : ring) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<W_MN>, mw, mx, a);
}

}  // namespace

cudaError_t launch_linear_rows(const mf_bf16* x, const mf_bf16* W, const TokenRuns& runs,
                               const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                               const LinearEpilogue& ep, const KernelCtl& ctl, cudaStream_t st) {
  return launch_rows<false>(x, W, runs, tok_mod, T, K, N, ep, ctl, st);
}

cudaError_t launch_linear_rows_dx(const mf_bf16* dz, const mf_bf16* W, const TokenRuns& runs,
                                  const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                                  mf_bf16* dx, const KernelCtl& ctl, cudaStream_t st) {
  LinearEpilogue ep{};
  ep.out = dx;
  return launch_rows<true>(dz, W, runs, tok_mod, T, K, N, ep, ctl, st);
}

}  // namespace mf
