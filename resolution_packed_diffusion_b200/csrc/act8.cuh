// act8.cuh -- device helpers of the 8-bit activation checkpoints (codes of eight
// channels travel as a uint2) and of the activations read through them.
#pragma once

#include <cstdint>

#include "mf_internal.h"
#include "mf_ptx.cuh"
#include "mlp_internal.h"

namespace mf {

__device__ __forceinline__ void bf16x8_unpack(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 bf16x8_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Four signed bytes as floats: byte b ^ 0x80 in the low mantissa bits of 2^23
// is 2^23 + b + 128, exactly; one byte permute and one subtraction a value, off
// the quarter-rate integer conversion path.
__device__ __forceinline__ void s8x4_float(uint32_t w, float* f) {
  const uint32_t u = w ^ 0x80808080u;
  f[0] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.f;
  f[1] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.f;
  f[2] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.f;
  f[3] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.f;
}

__device__ __forceinline__ void act8_load(const uint2& q, float s, float (&f)[8]) {
  s8x4_float(q.x, f);
  s8x4_float(q.y, f + 4);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= s;
}

// Scale and reciprocal step of a block whose largest |x| is `amax` (its bit
// pattern orders NaN above infinity above every number): amax / 127 and
// 127 / amax, both IEEE divisions; a block below 2^-100, whose reciprocal could
// overflow, is stored as zeros; one with a non-finite value gets the scale NaN,
// so that it reads back as NaN throughout instead of as wrong numbers.
__device__ __forceinline__ void act8_scale(float amax, float& s, float& inv) {
  const bool bad = !(amax <= 3.402823466e38f);
  const bool zero = amax < 7.888609052e-31f;
  s = bad ? __uint_as_float(0x7FC00000u) : (zero ? 0.f : __fdiv_rn(amax, 127.f));
  inv = bad || zero ? 0.f : __fdiv_rn(127.f, amax);
}

// Code of x under the reciprocal step inv (0 in a zero or non-finite block):
// round to nearest even of the rounded product, so |code| <= 127. Adding
// 1.5 * 2^23 leaves the integer in the low bits of the sum.
__device__ __forceinline__ uint32_t act8_code(float x, float inv) {
  const float p = inv == 0.f ? 0.f : __fmul_rn(x, inv);
  return __float_as_uint(__fadd_rn(p, 12582912.f)) & 0xFFu;
}

__device__ __forceinline__ uint32_t act8_code4(const float* x, float inv) {
  const uint32_t a = act8_code(x[0], inv), b = act8_code(x[1], inv), c = act8_code(x[2], inv),
                 d = act8_code(x[3], inv);
  return a | (b << 8) | (c << 16) | (d << 24);
}

// act(z) and act'(z). GELU, tanh form: 0.5 z (1 + tanh u) = z sigma(2u) with
// u = sqrt(2/pi) (z + 0.044715 z^3); SiLU: z sigma(z). Both are z sigma(w) with
// w = c1 z + c3 z^3, so act' = sigma + z sigma (1 - sigma) w'. sigma(w) =
// 1 / (1 + e^-w): e^-w overflows to infinity for large negative w, where the
// reciprocal is 0 as it should be, and 0 * z stays 0 for finite z.
struct ActValue {
  float f, d;
};
template <int ACT>
__device__ __forceinline__ float act_sigma(float z) {
  float w = z;
  if constexpr (ACT == MF_ACT_GELU) w = z * fmaf(0.07135481627f, z * z, 1.5957691216f);
  return __fdividef(1.f, 1.f + __expf(-w));
}
template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == MF_ACT_NONE) return z;
  return z * act_sigma<ACT>(z);
}
template <int ACT>
__device__ __forceinline__ float act_grad(float z) {
  if constexpr (ACT == MF_ACT_NONE) return 1.f;
  const float s = act_sigma<ACT>(z);
  float dw = 1.f;
  if constexpr (ACT == MF_ACT_GELU) dw = fmaf(0.2140644488f, z * z, 1.5957691216f);
  // past the saturation of sigma, z w' may overflow while its factor is 0
  const float t = s * (1.f - s);
  return t == 0.f ? s : fmaf(z * dw, t, s);
}

}  // namespace mf
