// act8.cuh -- device helpers of the 8-bit activation checkpoints (codes of eight
// channels travel as a uint2) and of the activations read through them.
#pragma once

#include <cstdint>

#include "mf_internal.h"
#include "mf_ptx.cuh"
#include "mlp_internal.h"

namespace mf {

// Values travel in pairs (f32x2 instructions: one for two values).
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }

__device__ __forceinline__ uint64_t bf16x2_f2(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t f2_bf16x2(uint64_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ void bf16x8_f2(const uint4& u, uint64_t (&f)[4]) {
  f[0] = bf16x2_f2(u.x);
  f[1] = bf16x2_f2(u.y);
  f[2] = bf16x2_f2(u.z);
  f[3] = bf16x2_f2(u.w);
}
__device__ __forceinline__ uint4 f2_bf16x8(const uint64_t (&f)[4]) {
  return make_uint4(f2_bf16x2(f[0]), f2_bf16x2(f[1]), f2_bf16x2(f[2]), f2_bf16x2(f[3]));
}

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

// Eight codes as numbers. Byte b ^ 0x80 in the low mantissa bits of 2^23 is
// 2^23 + b + 128, exactly: one byte permute a value and one subtraction a pair, off
// the quarter-rate integer conversion path.
__device__ __forceinline__ void act8_codes(const uint2& q, uint64_t (&f)[4]) {
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
  const uint64_t bias = f2_both(-8388736.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i >> 1];
    const uint32_t lo = __byte_perm(u, 0x4B000000u, (i & 1) ? 0x7442 : 0x7440);
    const uint32_t hi = __byte_perm(u, 0x4B000000u, (i & 1) ? 0x7443 : 0x7441);
    f[i] = f2_add(f2_pack(__uint_as_float(lo), __uint_as_float(hi)), bias);
  }
}

// Eight codes as the values they stand for.
__device__ __forceinline__ void act8_load(const uint2& q, float s, uint64_t (&f)[4]) {
  act8_codes(q, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_mul(f[i], f2_both(s));
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

// The same by a whole warp whose even and odd lanes share a block: one division a
// lane, exchanged.
__device__ __forceinline__ void act8_scale_pairwise(float amax, bool odd, float& s, float& inv) {
  const bool bad = !(amax <= 3.402823466e38f);
  const bool zero = amax < 7.888609052e-31f;
  const float a = bad || zero ? 1.f : amax;
  const float mine = __fdiv_rn(odd ? 127.f : a, odd ? a : 127.f);
  const float other = __shfl_xor_sync(0xffffffffu, mine, 1);
  s = bad ? __uint_as_float(0x7FC00000u) : (zero ? 0.f : (odd ? other : mine));
  inv = bad || zero ? 0.f : (odd ? mine : other);
}

// Four codes of (a.lo, a.hi, b.lo, b.hi) under the reciprocal step: round to nearest
// even of the rounded product, so |code| <= 127 (1.5 * 2^23 added, the integer is
// in the low bits of the sum). The products are scalar: the compiler contracts a
// packed product and sum to one rounding, which moves the ties at x = amax / 2.
// `mask` is 0 in a zero or non-finite block.
__device__ __forceinline__ uint32_t act8_code4(uint64_t a, uint64_t b, float inv, uint32_t mask) {
  const uint64_t round = f2_both(12582912.f);
  float c0, c1, c2, c3;
  f2_unpack(a, c0, c1);
  f2_unpack(b, c2, c3);
  f2_unpack(f2_add(f2_pack(__fmul_rn(c0, inv), __fmul_rn(c1, inv)), round), c0, c1);
  f2_unpack(f2_add(f2_pack(__fmul_rn(c2, inv), __fmul_rn(c3, inv)), round), c2, c3);
  const uint32_t lo = __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(c2), __float_as_uint(c3), 0x0040);
  return __byte_perm(lo, hi, 0x5410) & mask;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// act(z) and act'(z) of pairs. GELU, tanh form: 0.5 z (1 + tanh u) = z sigma(2u) with
// u = sqrt(2/pi) (z + 0.044715 z^3); SiLU: z sigma(z). Both are z sigma(w), w = c1 z +
// c3 z^3, so act' = sigma + z w' sigma (1 - sigma). sigma(w) = 1 / (1 + e), e = 2^v, v =
// -w log2(e); a pair shares one reciprocal, 1 / ((1 + a)(1 + b)), since two special
// functions a value already bound these kernels. 1 - sigma is taken as e sigma: where
// sigma is near 1, sigma - sigma^2 is the reciprocal's rounding and no more, and z w' of
// GELU, up to 5800, made it 7e-4 (measured). z is held at ActCoef::low, where act and act' are
// below 1e-16 in magnitude, so that the product cannot overflow (e < 2^62); act' holds it
// at 30 too, where e is 0. A NaN stays in its own lane: the shared reciprocal sees 2^62 in
// its place (a minimum with a number drops NaN), and the product with z makes that lane's
// result NaN again. BLOCK: values read back from a checkpoint, whose blocks are NaN
// throughout or not at all, go without the minimum (16384 x 12288 stored and read back
// through the GELU: 204.2 us, 207.8 with it).
template <int ACT>
struct ActCoef;
template <>
struct ActCoef<MF_ACT_GELU> {
  static constexpr float low = -7.5f;
  static constexpr float v1 = -2.302208198f, v3 = -0.1029432397f;  // -log2(e) (c1, c3)
  static constexpr float d1 = 1.5957691216f, d3 = 0.2140644488f;   // w' = c1 + 3 c3 z^2
};
template <>
struct ActCoef<MF_ACT_SILU> {
  static constexpr float low = -42.f;
  static constexpr float v1 = -1.442695041f, v3 = 0.f;
  static constexpr float d1 = 1.f, d3 = 0.f;
};

// sigma(w(z)), and e.
template <int ACT, bool BLOCK>
__device__ __forceinline__ uint64_t act_sigma2(uint64_t z, uint64_t zz, uint64_t& e) {
  using C = ActCoef<ACT>;
  const uint64_t v = ACT == MF_ACT_GELU
                         ? f2_mul(z, f2_fma(zz, f2_both(C::v3), f2_both(C::v1)))
                         : f2_mul(z, f2_both(C::v1));
  float a, b;
  f2_unpack(v, a, b);
  if constexpr (!BLOCK) {
    a = fminf(a, 62.f);
    b = fminf(b, 62.f);
  }
  e = f2_pack(ex2_approx(a), ex2_approx(b));
  f2_unpack(f2_add(e, f2_both(1.f)), a, b);
  const float r = rcp_approx(a * b);
  return f2_mul(f2_both(r), f2_pack(b, a));
}

template <int ACT, bool BLOCK = false>
__device__ __forceinline__ uint64_t act_fwd2(uint64_t z) {
  if constexpr (ACT == MF_ACT_NONE) return z;
  else {
    float a, b;
    uint64_t e;
    f2_unpack(z, a, b);
    z = f2_pack(max_nan(a, ActCoef<ACT>::low), max_nan(b, ActCoef<ACT>::low));
    return f2_mul(z, act_sigma2<ACT, BLOCK>(z, f2_mul(z, z), e));
  }
}

template <int ACT>
__device__ __forceinline__ uint64_t act_grad2(uint64_t z) {
  using C = ActCoef<ACT>;
  float a, b;
  uint64_t e;
  f2_unpack(z, a, b);
  z = f2_pack(min_nan(max_nan(a, C::low), 30.f), min_nan(max_nan(b, C::low), 30.f));
  const uint64_t zz = f2_mul(z, z);
  const uint64_t s = act_sigma2<ACT, false>(z, zz, e);
  uint64_t zd = z;  // z w'
  if constexpr (ACT == MF_ACT_GELU) zd = f2_mul(z, f2_fma(zz, f2_both(C::d3), f2_both(C::d1)));
  return f2_fma(zd, f2_mul(f2_mul(e, s), s), s);
}

// The checkpoint kernels: CTAs of 256 threads, sixteen lanes to a block of 128
// channels with eight each, or (WIDE) eight lanes with sixteen each, where every row
// starts on a 32-byte boundary of the bf16 tensor: half the loads, stores, shuffles
// and divisions a value (store and read back at 16384 x 12288: 217 -> 200 us).
// kAct8Unroll blocks per thread, all loads issued before the first is used.
constexpr int kAct8Threads = 256;
constexpr int kAct8Unroll = 4;
template <bool WIDE>
struct Act8Shape {
  static constexpr int PER_LANE = WIDE ? 16 : 8;
  static constexpr int LANES = kAct8Block / PER_LANE;
  static constexpr int PER_CTA = kAct8Threads / LANES;  // blocks a CTA takes per step
};
inline unsigned act8_ctas(uint32_t items, bool wide) {
  const uint32_t per = (wide ? Act8Shape<true>::PER_CTA : Act8Shape<false>::PER_CTA) * kAct8Unroll;
  return (items + per - 1) / per;
}
inline bool act8_wide(const void* bf16_rows, int32_t C) {
  return C % 16 == 0 && (reinterpret_cast<uintptr_t>(bf16_rows) & 31u) == 0;
}

// n / d for n < 2^31 by one high product (Granlund and Montgomery's method): with
// 2^shift >= d, mul = floor(2^32 (2^shift - d) / d) + 1, the quotient is
// (mulhi(mul, n) + n) >> shift.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {d, 0, 0};
  while ((1u << f.shift) < d) ++f.shift;
  f.mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << f.shift) - d)) / d + 1);
  return f;
}

// Where block `item` of the checkpoint lies: its row and first channel.
struct Act8Rows {
  FastDiv nb;      // blocks of a row
  int32_t C;
  uint32_t items;  // rows x blocks, below 2^31
};
// Rows of one launch, so that its items stay below 2^31.
inline int32_t act8_rows_max(int32_t C) { return 0x7FFFFFFF / act8_blocks(C); }
inline Act8Rows act8_rows(int32_t T, int32_t C) {
  const uint32_t nb = act8_blocks(C);
  return Act8Rows{fast_div(nb), C, static_cast<uint32_t>(T) * nb};
}

__device__ __forceinline__ void load_sector(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void store_sector(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// One CTA's share of y = act(q s).
template <int ACT, bool WIDE>
__device__ __forceinline__ void act8_decode(const int8_t* __restrict__ q,
                                            const float* __restrict__ scale, const Act8Rows& rows,
                                            mf_bf16* __restrict__ y, uint32_t block) {
  using S = Act8Shape<WIDE>;
  const int lane = threadIdx.x % S::LANES;
  const uint32_t base = block * (S::PER_CTA * kAct8Unroll) + threadIdx.x / S::LANES;
  uint4 v[kAct8Unroll];
  float s[kAct8Unroll];
  int64_t off[kAct8Unroll];
  bool in[kAct8Unroll];
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    const uint32_t item = base + u * S::PER_CTA;
    const uint32_t row = rows.nb.div(item);
    const int c = static_cast<int>(item - row * rows.nb.d) * kAct8Block + lane * S::PER_LANE;
    in[u] = item < rows.items && c < rows.C;
    off[u] = static_cast<int64_t>(row) * rows.C + c;
    v[u] = make_uint4(0, 0, 0, 0);
    if (in[u]) {
      if constexpr (WIDE) {
        v[u] = __ldcs(reinterpret_cast<const uint4*>(q + off[u]));
      } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(q + off[u]));
        v[u].x = w.x;
        v[u].y = w.y;
      }
    }
    s[u] = item < rows.items ? __ldg(scale + item) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kAct8Unroll; ++u) {
    uint64_t f[4], g[4];
    act8_load(make_uint2(v[u].x, v[u].y), s[u], f);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = act_fwd2<ACT, true>(f[e]);
    if constexpr (WIDE) {
      act8_load(make_uint2(v[u].z, v[u].w), s[u], g);
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = act_fwd2<ACT, true>(g[e]);
      if (in[u]) store_sector(y + off[u], f2_bf16x8(f), f2_bf16x8(g));
    } else {
      if (in[u]) __stcs(reinterpret_cast<uint4*>(y + off[u]), f2_bf16x8(f));
    }
  }
}

}  // namespace mf
