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
  uint16_t* v;             // fp16 [M][rp]: scaling * x . A^T of the row, over unit[m]
  float* unit;             // [M]: a power of two
  int* status;
  int M, K, N, r, adapters;
  int rp;                  // r rounded up to 16
  int splits;              // CTAs of a cluster, each a part of K (first product)
  int passes;              // CTAs that share the adapters of a block of rows (first product)
  int groups;              // the same for the second product
};

constexpr int kLoraMaxRank = 128;

// Fills splits, passes and groups.
void lora_plan(LoraParams* p, int sms);
cudaError_t launch_lora_down(const LoraParams& p, cudaStream_t stream);
cudaError_t launch_lora_up(const LoraParams& p, cudaStream_t stream);

}  // namespace w4a16
