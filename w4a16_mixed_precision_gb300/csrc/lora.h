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
  uint16_t* v;             // workspace, for many rows: fp16 [M][rp], scaling * x . A^T of the row over unit[m]
  float* unit;             // workspace: [M], a power of two
  int* arrived;            // workspace: warps done with each 128 rows; like v and unit zero between calls
  int rp;                  // r rounded up to 16
  int* status;
  int M, K, N, r, adapters;
  int splits;              // CTAs of a cluster (filled in by launch_lora, like shares)
  int shares;              // clusters at most that share the columns of an item
};

constexpr int kLoraMaxRank = 128;

// half: 0 the first product, 1 the second; where lora_two_kernels is false half 0
// is not launched and half 1 does both.
bool lora_two_kernels(int M, int r);
cudaError_t launch_lora(LoraParams p, int half, int sms, cudaStream_t stream);

}  // namespace w4a16
