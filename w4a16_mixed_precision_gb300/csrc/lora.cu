// lora.cu -- low-rank adapters of many requests beside a shared product:
//     y[m] += scaling[a] * (x[m] . A[a]^T) . B[a]^T,   a = index[m] (none if negative),
// A[a] r x K and B[a] N x r in fp16.  Two kernels: down (v = x . A^T, fp32,
// split over K) and up (y += v . B^T).
//
// Bound: for few rows reading the adapters in use, r (K + N) fp16 each; for
// many rows reading x and reading and writing y, and the matrix instructions.
//   * Rows are taken in blocks of 16 or 32.  A block makes one pass for each
//     different adapter among its rows (one, for the rows of a prompt), with the
//     other rows' operand zeroed, so any order of rows is right and runs of
//     equal adapters are fast.  Which rows share an adapter is found in the
//     kernel by a vote; for small batches the passes of a block go to
//     different CTAs.
//   * mma.sync with the rows as the 16-row operand.  The k order is permuted
//     alike in both operands so that every lane loads 16 consecutive bytes.
//   * v is scaled, normalised by a power of two per row (so that no magnitude
//     of x leaves fp16's range) and rounded to fp16 for the second product: one
//     rounding of 2^-12 per term of a sum that is itself an addition to y.
#include "lora.h"

#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kWarps = 4;
constexpr int kLoraSite = 104;  // the word after the status word: an adapter index out of range

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The adapters of a block of up to 32 rows, one row per lane.
struct Block {
  int mine;          // this lane's row's adapter, -1 for none
  uint32_t leaders;  // the first row of each different adapter
  int pass;          // which of them this lane's row belongs to
};

__device__ __forceinline__ Block block_adapters(const LoraParams& p, int row0, int rows) {
  const int lane = threadIdx.x & 31;
  Block k;
  k.mine = lane < rows && row0 + lane < p.M ? p.index[row0 + lane] : -1;
  if (k.mine >= p.adapters) {
    atomicCAS(p.status + 1, 0, kLoraSite);
    atomicOr(p.status, kStatusBounds);
    k.mine = -1;
  }
  if (k.mine < 0) k.mine = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, k.mine);
  const int first = __ffs(same) - 1;
  k.leaders = __ballot_sync(0xffffffffu, k.mine >= 0 && lane == first);
  k.pass = k.mine < 0 ? -1 : __popc(k.leaders & ((1u << first) - 1));
  return k;
}

// v[split][m][j] of the rows whose pass is one of this CTA's.  MT: 16-row tiles
// per block; NT: 8-rank tiles per CTA.
template <int MT, int NT>
__global__ void __launch_bounds__(kWarps * 32) lora_down_kernel(const LoraParams p) {
  __shared__ float red[kWarps][16 * MT][NT * 8 + 1];
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int chunks = (p.r + NT * 8 - 1) / (NT * 8);
  const int row0 = (blockIdx.x / chunks) * (16 * MT), j0 = (blockIdx.x % chunks) * (NT * 8);
  const Block k = block_adapters(p, row0, 16 * MT);
  const int count = __popc(k.leaders);
  if ((int)blockIdx.z >= count) return;

  // this warp's 32-wide K steps
  const int steps = p.K / 32, parts = p.splits * kWarps, part = blockIdx.y * kWarps + warp;
  const int s0 = (int)((long long)steps * part / parts), s1 = (int)((long long)steps * (part + 1) / parts);

  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;

  uint32_t left = k.leaders;
  for (int pass = 0; pass < count; ++pass, left &= left - 1) {
    if (pass % p.passes != (int)blockIdx.z) continue;
    const int ad = __shfl_sync(0xffffffffu, k.mine, __ffs(left) - 1);
    const uint32_t rows = __ballot_sync(0xffffffffu, k.mine == ad);
    const uint16_t* a = p.a + ((long long)ad * p.r + j0) * p.K + c * 8;
    const uint16_t* x = p.x + (long long)row0 * p.K + c * 8;
#pragma unroll 2
    for (int s = s0; s < s1; ++s) {
      uint4 xr[MT][2], ar[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        ar[j] = j0 + j * 8 + g < p.r ? __ldg(reinterpret_cast<const uint4*>(a + (long long)(j * 8 + g) * p.K + s * 32))
                                     : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * i + 8 * e + g;
          xr[i][e] = (rows >> row) & 1u ? *reinterpret_cast<const uint4*>(x + (long long)row * p.K + s * 32)
                                        : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816(acc[i][j], xr[i][0].x, xr[i][1].x, xr[i][0].y, xr[i][1].y, ar[j].x, ar[j].y);
          mma16816(acc[i][j], xr[i][0].z, xr[i][1].z, xr[i][0].w, xr[i][1].w, ar[j].z, ar[j].w);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[warp][16 * i + g + 8 * (e >> 1)][j * 8 + 2 * c + (e & 1)] = acc[i][j][e];
  __syncthreads();
  for (int t = threadIdx.x; t < 16 * MT * NT * 8; t += kWarps * 32) {
    const int row = t / (NT * 8), j = t - row * (NT * 8);  // row is the same in a warp where NT * 8 >= 32
    const int pass = __shfl_sync(0xffffffffu, k.pass, row);
    if (pass < 0 || pass % p.passes != (int)blockIdx.z || j0 + j >= p.r) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w][row][j];
    p.v[((long long)blockIdx.y * p.M + row0 + row) * p.r + j0 + j] = sum;
  }
}

// y += scaling v . B^T for the rows whose pass is one of this CTA's; every warp
// takes 32 columns of the CTA's 128.
template <int MT>
__global__ void __launch_bounds__(kWarps * 32) lora_up_kernel(const LoraParams p) {
  __shared__ __half vh[16 * MT][kLoraMaxRank + 8];
  __shared__ float unit[16 * MT];
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * (16 * MT), n0 = blockIdx.y * (kWarps * 32) + warp * 32;
  griddep_wait();
  const Block k = block_adapters(p, row0, 16 * MT);
  const int count = __popc(k.leaders);
  if ((int)blockIdx.z >= count) return;

  // v of this CTA's rows: sum of the K splits in order, scaled, as fp16
  const int rp = (p.r + 15) / 16 * 16;
  for (int row = warp; row < 16 * MT; row += kWarps) {
    const int pass = __shfl_sync(0xffffffffu, k.pass, row), ad = __shfl_sync(0xffffffffu, k.mine, row);
    const bool on = pass >= 0 && pass % p.passes == (int)blockIdx.z;
    float s[kLoraMaxRank / 32], top = 0.f;
#pragma unroll
    for (int i = 0; i < kLoraMaxRank / 32; ++i) {
      const int j = 32 * i + lane;
      s[i] = 0.f;
      if (on && j < p.r) {
        for (int q = 0; q < p.splits; ++q) s[i] += p.v[((long long)q * p.M + row0 + row) * p.r + j];
        s[i] *= p.scaling[ad];
      }
      top = fmaxf(top, fabsf(s[i]));
    }
#pragma unroll
    for (int q = 1; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
    // 2^exponent of the row's largest magnitude
    const float u = top > 1e-30f ? __uint_as_float(__float_as_uint(top) & 0x7F800000u) : 1.f;
#pragma unroll
    for (int i = 0; i < kLoraMaxRank / 32; ++i)
      if (32 * i + lane < rp) vh[row][32 * i + lane] = __float2half_rn(s[i] / u);
    if (lane == 0) unit[row] = u;
  }
  __syncthreads();

  float acc[MT][4][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.f;
  uint32_t left = k.leaders;
  for (int pass = 0; pass < count; ++pass, left &= left - 1) {
    if (pass % p.passes != (int)blockIdx.z) continue;
    const int ad = __shfl_sync(0xffffffffu, k.mine, __ffs(left) - 1);
    const uint32_t rows = __ballot_sync(0xffffffffu, k.mine == ad);
    // operand column g of tile t is output column 8 (g / 2) + 2 t + g % 2 of the
    // warp's 32, so that a lane's results are 8 consecutive columns of y
    const uint16_t* b = p.b + ((long long)ad * p.N + n0 + 8 * (g >> 1) + (g & 1)) * p.r + 4 * c;
#pragma unroll 2
    for (int s = 0; s < rp; s += 16) {
      uint2 br[4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
        br[t] = s + 4 * c < p.r ? __ldg(reinterpret_cast<const uint2*>(b + (long long)(2 * t) * p.r + s))
                                : make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint2 v0 = *reinterpret_cast<const uint2*>(&vh[16 * i + g][s + 4 * c]);
        uint2 v1 = *reinterpret_cast<const uint2*>(&vh[16 * i + g + 8][s + 4 * c]);
        if (!((rows >> (16 * i + g)) & 1u)) v0 = make_uint2(0u, 0u);
        if (!((rows >> (16 * i + g + 8)) & 1u)) v1 = make_uint2(0u, 0u);
#pragma unroll
        for (int t = 0; t < 4; ++t) mma16816(acc[i][t], v0.x, v1.x, v0.y, v1.y, br[t].x, br[t].y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 16 * i + 8 * e + g;
      const int pass = __shfl_sync(0xffffffffu, k.pass, row);
      if (pass < 0 || pass % p.passes != (int)blockIdx.z) continue;
      uint4* yp = reinterpret_cast<uint4*>(p.y + (long long)(row0 + row) * p.N + n0 + 8 * c);
      uint4 y = *yp;
      uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
      const float u = unit[row];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&yw[t]));
        const __half2 h = __floats2half2_rn(fmaf(acc[i][t][2 * e], u, f.x), fmaf(acc[i][t][2 * e + 1], u, f.y));
        yw[t] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *yp = y;
    }
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Blocks of 32 rows from 128 rows on: enough blocks to fill the card, and each
// adapter operand is used for twice as many rows.
int row_tiles(int M) { return M >= 128 ? 2 : 1; }

}  // namespace

void lora_plan(int M, int K, int adapters, int sms, int* splits, int* passes) {
  const int rows = 16 * row_tiles(M), blocks = (M + rows - 1) / rows;
  int most = M < rows ? M : rows;
  if (adapters < most) most = adapters;
  *passes = M >= 128 ? 1 : (most < 1 ? 1 : most);
  int s = (3 * sms) / (blocks * *passes);
  const int room = K / (32 * kWarps);  // a 32-wide step per warp at least
  if (s > room) s = room;
  if (s > kLoraMaxSplits) s = kLoraMaxSplits;
  *splits = s < 1 ? 1 : s;
}

cudaError_t launch_lora_down(const LoraParams& p, cudaStream_t stream) {
  const int mt = row_tiles(p.M), nt = p.r <= 8 ? 1 : p.r <= 16 ? 2 : p.r <= 32 ? 4 : 8;
  const int blocks = (p.M + 16 * mt - 1) / (16 * mt), chunks = (p.r + nt * 8 - 1) / (nt * 8);
  const dim3 grid(blocks * chunks, p.splits, p.passes);
#define W4A16_DOWN(MT, NT) \
  if (mt == MT && nt == NT) return launch(lora_down_kernel<MT, NT>, grid, p, stream);
  W4A16_DOWN(1, 1) W4A16_DOWN(1, 2) W4A16_DOWN(1, 4) W4A16_DOWN(1, 8)
  W4A16_DOWN(2, 1) W4A16_DOWN(2, 2) W4A16_DOWN(2, 4) W4A16_DOWN(2, 8)
#undef W4A16_DOWN
  return cudaErrorInvalidValue;
}

cudaError_t launch_lora_up(const LoraParams& p, cudaStream_t stream) {
  const int mt = row_tiles(p.M), blocks = (p.M + 16 * mt - 1) / (16 * mt);
  const dim3 grid(blocks, p.N / (kWarps * 32), p.passes);
  return mt == 1 ? launch(lora_up_kernel<1>, grid, p, stream) : launch(lora_up_kernel<2>, grid, p, stream);
}

}  // namespace w4a16
