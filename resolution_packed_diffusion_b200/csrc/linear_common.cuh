// linear_common.cuh -- what the two kernels of the fused linear layer share: tensor
// maps, the bounded drain, TMEM reads.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "act8.cuh"
#include "mf_ptx.cuh"
#include "mlp_internal.h"

namespace mf {

// The same value in every lane, told to the compiler.
__device__ __forceinline__ int warp_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint32_t warp_uniform(uint32_t v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// umma_ss / umma_ss_pair and their commits for a warp that issues as one: every lane
// runs the loop, so that descriptors and addresses live in uniform registers, and
// `leader` (true in one lane, always the same) issues.
__device__ __forceinline__ void umma_ss_by(bool leader, uint32_t d_tmem, uint64_t adesc,
                                           uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void umma_ss_pair_by(bool leader, uint32_t d_tmem, uint64_t adesc,
                                                uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void umma_commit_by(bool leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void umma_commit_pair_by(bool leader, uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"(mask), "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// The producer's copies and byte counts in the same manner.
__device__ __forceinline__ void load_2d_by(bool leader, void* dst, const CUtensorMap* map,
                                           uint64_t* bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void load_2d_pair_by(bool leader, void* dst, const CUtensorMap* map,
                                                uint32_t leader_bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}
__device__ __forceinline__ void expect_by(bool leader, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// L2 policy of the weights, which every row block reads again.
__device__ __forceinline__ uint64_t keep_in_l2() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Waits for copies or MMAs in flight before their shared memory is used otherwise or the
// CTA leaves. At least 50 ms, however short the limit of the other waits: a copy that
// lands after its CTA has left writes to memory that is someone else's.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  constexpr uint64_t kLeastNs = 50000000ull;
  const uint64_t limit = limit_ns > kLeastNs ? limit_ns : kLeastNs;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit) return;
}

// 32 columns of one accumulator row; the caller masks what it stores.
__device__ __forceinline__ void acc_load32(uint32_t taddr, float (&f)[32]) {
  uint32_t v[32];
  tmem_ld32(taddr, v);
  tmem_ld_wait();
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    asm volatile("" : "+r"(v[e]));
    f[e] = __uint_as_float(v[e]);
  }
}

// [sets][rows][cols] bf16 with boxes of 64 columns x box_rows, 128-byte swizzle; what
// lies outside reads as zeros. sets 0: a two-dimensional map.
bool linear_map(CUtensorMap* map, const mf_bf16* base, int64_t cols, int64_t rows, int sets,
                int box_rows);

// Few rows (linear_rows.cu): the forward, and dx. The border is the N of that kernel's
// MMAs. It is not where the two kernels cost the same: at 128 rows, 3072 -> 12288 takes
// 26.7 us here and 21.8 in tiles at 129 (dx 21.9 and 51.8), 12288 -> 3072 takes 23.2 here
// and 54.2 in tiles (dx 22.8 and 22.8). In tiles an inner dimension of 12288 is walked by
// 48 pairs of SMs, 192 steps each.
constexpr int kFewRows = 128;
inline bool few_rows(int32_t T) { return T <= kFewRows; }
cudaError_t launch_linear_rows(const mf_bf16* x, const mf_bf16* W, const TokenRuns& runs,
                               const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                               const LinearEpilogue& ep, const KernelCtl& ctl, cudaStream_t st);
cudaError_t launch_linear_rows_dx(const mf_bf16* dz, const mf_bf16* W, const TokenRuns& runs,
                                  const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                                  mf_bf16* dx, const KernelCtl& ctl, cudaStream_t st);

}  // namespace mf
