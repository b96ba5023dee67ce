// lora.h -- internal interface of the low-rank adapter kernels (lora.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace w4a16 {

struct LoraParams {
  const uint16_t* x;       // fp16 [M][K]
  const uint16_t* a;       // fp16 [adapters][r][K]
  const uint16_t* b;       // fp16 [adapters][N][r]
  const float* scaling;    // [adapters]
  const int* index;        // [M]: the row's adapter, negative for none
  uint16_t* y;             // fp16 [M][N], the base product; the adapters' part is added to it
  float* v;                // fp32 [splits][M][r]: x . A^T, a partial sum per K split
  int* status;
  int M, K, N, r, adapters;
  int splits;              // K splits of the first product
  int passes;              // CTAs that share the adapters of a block of rows
};

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxSplits = 16;

// K splits and CTAs per block of rows for this problem.
void lora_plan(int M, int K, int adapters, int sms, int* splits, int* passes);
cudaError_t launch_lora_down(const LoraParams& p, cudaStream_t stream);
cudaError_t launch_lora_up(const LoraParams& p, cudaStream_t stream);

}  // namespace w4a16
