// mlp_internal.h -- launchers of the MLP-branch operators: the modality-specific
// layer norm (layer_norm.cu), activation checkpoints in 8 bits (act8.cu) and the
// fused linear layer (linear_fused.cu). Not part of the public ABI (include/mf.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime_api.h>

#include "mf_internal.h"

namespace mf {

constexpr int kAct8Block = MF_ACT8_BLOCK;  // channels that share one scale
inline int32_t act8_blocks(int32_t C) { return (C + kAct8Block - 1) / kAct8Block; }

// One 8-bit checkpoint of a [T][C] activation: codes [T][C], scales [T][act8_blocks(C)].
struct Act8 {
  const int8_t* q;
  const float* scale;
};

cudaError_t launch_act8_quantize(const mf_bf16* x, int32_t T, int32_t C, int8_t* q, float* scale,
                                 cudaStream_t st);
cudaError_t launch_act8_dequantize(const int8_t* q, const float* scale, int32_t T, int32_t C,
                                   int32_t act, mf_bf16* y, cudaStream_t st);

// stats may be NULL.
cudaError_t launch_layer_norm(const mf_bf16* x, const float* gamma, const float* beta,
                              const uint8_t* tok_mod, int32_t T, int32_t hid, float eps,
                              mf_bf16* y, float* stats, const KernelCtl& ctl, cudaStream_t st);
// Bytes of the column sums' partials; x or x8 gives the forward's input.
size_t layer_norm_bwd_ws(int32_t T, int32_t hid);
cudaError_t launch_layer_norm_bwd(const mf_bf16* dy, const mf_bf16* x, const Act8& x8,
                                  const float* gamma, const float* stats, const uint8_t* tok_mod,
                                  const mf_bf16* resid, int32_t T, int32_t hid, mf_bf16* dx,
                                  float* dgamma, float* dbeta, void* ws, const KernelCtl& ctl,
                                  cudaStream_t st);

// Rows of each modality as runs of consecutive tokens (a sample's image tokens,
// then its text tokens; neighbouring runs of one modality are one run).
struct TokenRuns {
  int32_t n[2];
  int32_t count[2];  // tokens of the modality
  int32_t start[2][MF_MAX_SAMPLES];
  int32_t len[2][MF_MAX_SAMPLES];
};
// false if the descriptors are invalid (negative sizes, more than MF_MAX_TOKENS).
bool token_runs(const mf_sample_desc* desc, int32_t S, TokenRuns* runs, int32_t* T);

// Epilogue of the fused linear layer; every pointer but out may be NULL.
struct LinearEpilogue {
  const float* bias;     // [2][N]
  const mf_bf16* resid;  // [T][N]
  mf_bf16* z;            // [T][N], the pre-activation
  int8_t* z8;            // [T][N] with z_scale [T][act8_blocks(N)]
  float* z_scale;
  mf_bf16* out;
  int32_t act;
};
cudaError_t launch_linear_fused(const mf_bf16* x, const mf_bf16* W, const TokenRuns& runs,
                                const uint8_t* tok_mod, int32_t T, int32_t K, int32_t N,
                                const LinearEpilogue& ep, const KernelCtl& ctl, cudaStream_t st);

struct LinearBwd {
  const mf_bf16* dout;   // [T][N]
  const mf_bf16* x;      // [T][K], or x8
  Act8 x8;
  const mf_bf16* W;      // [2][N][K]
  const mf_bf16* z;      // [T][N], or z8 (act != none)
  Act8 z8;
  const uint8_t* tok_mod;
  int32_t act;
  mf_bf16* dx;           // any of the three may be NULL
  mf_bf16* dW;
  float* db;
};
size_t linear_fused_bwd_ws(int32_t T, int32_t K, int32_t N);
cudaError_t launch_linear_fused_bwd(const LinearBwd& b, const TokenRuns& runs, int32_t T, int32_t K,
                                    int32_t N, void* ws, const KernelCtl& ctl, cudaStream_t st);

}  // namespace mf
