// act8.cu -- activation checkpoints in 8 bits: a [T][C] bf16 activation kept for
// the backward as int8 codes with one fp32 scale per token and 128 channels,
//   s = amax / 127, q = rint(x * (127 / amax)), x ~ q s,
// and read back through the activation that followed it, y = act(q s).
//
// Why this form: the error of a code is at most s / 2 = amax / 254, relative RMS
// about 0.6% for a normal block (an 8-bit float with three mantissa bits has
// 2.6%); 128 channels keep one outlier from costing a whole row its precision at
// 3% extra bytes. The picx.dev "Mage-Flow" summary (Methodology > Training
// Infrastructure) names training under a memory budget; the format is this
// library's own.
//
// Both kernels are bound by HBM (3 bytes a value plus the scales). At 16384 x 3072, sixteen
// channels a lane: 25.1 us stored (0.93 of it), 24.2 us read back (0.96), 27.0 through the
// GELU (0.86). A block's lanes find its maximum by shuffles and share its two divisions
// (act8.cuh).
#include <cuda_bf16.h>

#include <cstdint>

#include "act8.cuh"
#include "mlp_internal.h"
#include "pdl.cuh"

namespace mf {

namespace {

// Largest |x| of eight bf16 values as a 15-bit pattern (NaN above infinity).
__device__ __forceinline__ uint32_t absmax_bits(const uint4& u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                              __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

template <bool WIDE>
__global__ void __launch_bounds__(kAct8Threads)
    act8_quantize_kernel(const mf_bf16* __restrict__ x, const Act8Rows rows,
                         int8_t* __restrict__ q, float* __restrict__ scale) {
  using S = Act8Shape<WIDE>;
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x % S::LANES;
  const uint32_t base = blockIdx.x * (S::PER_CTA * kAct8Unroll) + threadIdx.x / S::LANES;
  uint4 v[kAct8Unroll], w[kAct8Unroll];
  int64_t off[kAct8Unroll];
  bool in[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const uint32_t item = base + u * S::PER_CTA;
    const uint32_t row = rows.nb.div(item);
    const int c = static_cast<int>(item - row * rows.nb.d) * kAct8Block + lane * S::PER_LANE;
    in[u] = item < rows.items && c < rows.C;
    off[u] = static_cast<int64_t>(row) * rows.C + c;
    v[u] = w[u] = make_uint4(0, 0, 0, 0);
    if (in[u]) {
      if constexpr (WIDE)
        load_sector(x + off[u], v[u], w[u]);
      else
        v[u] = __ldcs(reinterpret_cast<const uint4*>(x + off[u]));
    }
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    uint32_t m = absmax_bits(v[u]);
    if constexpr (WIDE) m = max(m, absmax_bits(w[u]));
#pragma unroll
    for (int o = S::LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s, inv;
    uint64_t f[4];
    act8_scale_pairwise(__uint_as_float(m << 16), lane & 1, s, inv);
    const uint32_t mask = inv == 0.f ? 0u : 0xFFFFFFFFu;
    bf16x8_f2(v[u], f);
    const uint2 a = make_uint2(act8_code4(f[0], f[1], inv, mask), act8_code4(f[2], f[3], inv, mask));
    if constexpr (WIDE) {
      bf16x8_f2(w[u], f);
      const uint2 b = make_uint2(act8_code4(f[0], f[1], inv, mask), act8_code4(f[2], f[3], inv, mask));
      if (in[u]) __stcs(reinterpret_cast<uint4*>(q + off[u]), make_uint4(a.x, a.y, b.x, b.y));
    } else {
      if (in[u]) __stcs(reinterpret_cast<uint2*>(q + off[u]), a);
    }
    const uint32_t item = base + u * S::PER_CTA;
    if (lane == 0 && item < rows.items) scale[item] = s;
  }
}

template <int ACT, bool WIDE>
__global__ void __launch_bounds__(kAct8Threads)
    act8_dequantize_kernel(const int8_t* __restrict__ q, const float* __restrict__ scale,
                           const Act8Rows rows, mf_bf16* __restrict__ y) {
  pdl_wait();
  pdl_release();
  act8_decode<ACT, WIDE>(q, scale, rows, y, blockIdx.x);
}

}  // namespace

cudaError_t launch_act8_quantize(const mf_bf16* x, int32_t T, int32_t C, int8_t* q, float* scale,
                                 cudaStream_t st) {
  const bool wide = act8_wide(x, C);
  auto kernel = wide ? act8_quantize_kernel<true> : act8_quantize_kernel<false>;
  for (int32_t t = 0, n; t < T; t += n) {
    n = T - t < act8_rows_max(C) ? T - t : act8_rows_max(C);
    const Act8Rows rows = act8_rows(n, C);
    const cudaError_t e = launch_dependent(
        kernel, dim3(act8_ctas(rows.items, wide)), dim3(kAct8Threads), 0, st,
        x + static_cast<size_t>(t) * C, rows, q + static_cast<size_t>(t) * C,
        scale + static_cast<size_t>(t) * act8_blocks(C));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_act8_dequantize(const int8_t* q, const float* scale, int32_t T, int32_t C,
                                   int32_t act, mf_bf16* y, cudaStream_t st) {
  const bool wide = act8_wide(y, C);
  auto kernel =
      act == MF_ACT_GELU
          ? (wide ? act8_dequantize_kernel<MF_ACT_GELU, true> : act8_dequantize_kernel<MF_ACT_GELU, false>)
      : act == MF_ACT_SILU
          ? (wide ? act8_dequantize_kernel<MF_ACT_SILU, true> : act8_dequantize_kernel<MF_ACT_SILU, false>)
          : (wide ? act8_dequantize_kernel<MF_ACT_NONE, true> : act8_dequantize_kernel<MF_ACT_NONE, false>);
  for (int32_t t = 0, n; t < T; t += n) {
    n = T - t < act8_rows_max(C) ? T - t : act8_rows_max(C);
    const Act8Rows rows = act8_rows(n, C);
    const cudaError_t e = launch_dependent(
        kernel, dim3(act8_ctas(rows.items, wide)), dim3(kAct8Threads), 0, st,
        q + static_cast<size_t>(t) * C, scale + static_cast<size_t>(t) * act8_blocks(C), rows,
        y + static_cast<size_t>(t) * C);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mf
