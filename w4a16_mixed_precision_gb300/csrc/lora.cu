// lora.cu -- low-rank adapters of many requests beside a shared product:
//     y[m] += scaling[a] * (x[m] . A[a]^T) . B[a]^T,   a = index[m] (none if negative),
// A[a] r x K and B[a] N x r in fp16.  Two kernels: down (v = scaling x . A^T) and
// up (y += v . B^T).
//
// Bound: for few rows reading the adapters in use, r (K + N) fp16 each; for
// many rows reading x, and reading and writing y.
//   * Rows are taken in blocks of 16 or 32.  A block makes one pass for each
//     different adapter among its rows (one, for the rows of a prompt), with the
//     other rows' operand zeroed, so any order of rows is right and runs of
//     equal adapters are fast.  Which rows share an adapter is found in the
//     kernel by a vote; for small batches the passes of a block go to
//     different CTAs.
//   * mma.sync with the rows as the 16-row operand.  The k order is permuted
//     alike in both operands so that every lane loads 16 consecutive bytes.
//   * down splits K over the warps of a CTA and the CTAs of a cluster, whose sums
//     meet in the first CTA's shared memory in a fixed order: no partial sums in
//     global memory and no second reduction.
//   * v is scaled, normalised by a power of two per row (so that no magnitude
//     of x leaves fp16's range) and rounded to fp16 for the second product: one
//     rounding of 2^-12 per term of a sum that is itself an addition to y.
#include "lora.h"

#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kDownWarps = 8;
constexpr int kUpWarps = 4;
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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The fp32 value at this CTA-local shared address in CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %1, %2;\n\tld.shared::cluster.f32 %0, [ra];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// v and unit of the rows whose pass is one of this cluster's.  MT: 16-row tiles
// per block; NT: 8-rank tiles (r <= 8 NT).  CTA rank in the cluster: the part of K.
template <int MT, int NT>
__global__ void __launch_bounds__(kDownWarps * 32) lora_down_kernel(const LoraParams p) {
  constexpr int kRows = 16 * MT, kRanks = 8 * NT, kAcc = MT * NT * 4;
  // half of the warps leave their sums to the other half, three times; then the CTA's sum
  __shared__ float red[kDownWarps / 2][kAcc][32];
  __shared__ float total[kRows][kRanks + 1];
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * kRows;
  const Block k = block_adapters(p, row0, kRows);
  const int count = __popc(k.leaders);
  if ((int)blockIdx.z >= count) return;  // alike in all CTAs of the cluster

  // this warp's 32-wide K steps
  const int steps = p.K / 32, parts = p.splits * kDownWarps, part = blockIdx.y * kDownWarps + warp;
  const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;

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
    const uint16_t* a = p.a + (long long)ad * p.r * p.K + c * 8;
    const uint16_t* x = p.x + (long long)row0 * p.K + c * 8;
    constexpr int kTogether = 2 * MT + NT <= 4 ? 4 : 2 * MT + NT <= 8 ? 2 : 1;  // steps whose loads go out together
#pragma unroll kTogether
    for (int s = s0; s < s1; ++s) {
      uint4 xr[MT][2], ar[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        ar[j] = j * 8 + g < p.r ? __ldg(reinterpret_cast<const uint4*>(a + (long long)(j * 8 + g) * p.K + s * 32))
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
  // ---- the sum over the warps, then over the cluster's CTAs, each in order -------------
#pragma unroll
  for (int half = kDownWarps / 2; half >= 1; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int t = 0; t < kAcc; ++t) red[warp - half][t][lane] = acc[t / (NT * 4)][t / 4 % NT][t % 4];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int t = 0; t < kAcc; ++t) acc[t / (NT * 4)][t / 4 % NT][t % 4] += red[warp][t][lane];
    }
    __syncthreads();
  }
  if (warp == 0) {
#pragma unroll
    for (int t = 0; t < kAcc; ++t) {
      const int i = t / (NT * 4), j = t / 4 % NT, e = t % 4;
      total[16 * i + g + 8 * (e >> 1)][8 * j + 2 * c + (e & 1)] = acc[i][j][e];
    }
  }
  if (p.splits > 1) cluster_sync();
  else __syncthreads();
  if (blockIdx.y == 0) {
    for (int row = warp; row < kRows; row += kDownWarps) {
      const int pass = __shfl_sync(0xffffffffu, k.pass, row), ad = __shfl_sync(0xffffffffu, k.mine, row);
      if (pass < 0 || pass % p.passes != (int)blockIdx.z) continue;
      const float scaling = p.scaling[ad];
      float s[(kRanks + 31) / 32], top = 0.f;
#pragma unroll
      for (int i = 0; i < (kRanks + 31) / 32; ++i) {
        const int j = 32 * i + lane;
        s[i] = 0.f;
        if (j < p.r) {
          s[i] = total[row][j];
          for (int q = 1; q < p.splits; ++q) s[i] += ld_cluster(smem_addr(&total[row][j]), (uint32_t)q);
          s[i] *= scaling;
        }
        top = fmaxf(top, fabsf(s[i]));
      }
#pragma unroll
      for (int q = 1; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
      // 2^exponent of the row's largest magnitude
      const float u = top > 1e-30f ? __uint_as_float(__float_as_uint(top) & 0x7F800000u) : 1.f;
#pragma unroll
      for (int i = 0; i < (kRanks + 31) / 32; ++i) {
        const int j = 32 * i + lane;
        if (j < p.rp) p.v[(long long)(row0 + row) * p.rp + j] = __half_as_ushort(__float2half_rn(s[i] / u));
      }
      if (lane == 0) p.unit[row0 + row] = u;
    }
  }
  if (p.splits > 1) cluster_sync();  // the sums stay until they are read
}

// y += v . B^T for the rows whose pass is one of this CTA's; every warp takes 32
// columns of the CTA's 128.
template <int MT>
__global__ void __launch_bounds__(kUpWarps * 32) lora_up_kernel(const LoraParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * (16 * MT), n0 = blockIdx.y * (kUpWarps * 32) + warp * 32;
  griddep_wait();
  const Block k = block_adapters(p, row0, 16 * MT);
  const int count = __popc(k.leaders);
  if ((int)blockIdx.z >= count) return;

  // this lane's pieces of y: rows g and g + 8 of each tile, columns 8c .. 8c + 7
  uint4 y[MT][2];
  float unit[MT][2];
  bool mine[MT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = 16 * i + 8 * e + g;
      const int pass = __shfl_sync(0xffffffffu, k.pass, row);
      mine[i][e] = pass >= 0 && pass % p.groups == (int)blockIdx.z;
      y[i][e] = make_uint4(0u, 0u, 0u, 0u);
      unit[i][e] = 0.f;
      if (mine[i][e]) {
        y[i][e] = *reinterpret_cast<const uint4*>(p.y + (long long)(row0 + row) * p.N + n0 + 8 * c);
        unit[i][e] = p.unit[row0 + row];
      }
    }

  float acc[MT][4][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][t][e] = 0.f;
  // operand column g of tile t is output column 8 (g / 2) + 2 t + g % 2 of the
  // warp's 32, so that a lane's results are 8 consecutive columns of y
  const uint16_t* b0 = p.b + (long long)(n0 + 8 * (g >> 1) + (g & 1)) * p.r + 4 * c;
  const int steps = p.rp / 16;
  // (pass, step) pairs, several at a time so that their loads are in flight together
  int pass = blockIdx.z, step = 0;
  uint32_t left = k.leaders;
  for (int q = 0; q < pass; ++q) left &= left - 1;
  constexpr int kAhead = 4;
  while (pass < count) {
    uint2 br[kAhead][4], v[kAhead][MT][2];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const bool on = pass < count;
      const int ad = __shfl_sync(0xffffffffu, k.mine, on ? __ffs(left) - 1 : 0);
      const uint32_t rows = on ? __ballot_sync(0xffffffffu, k.mine == ad) : 0u;
      const bool in = on && 16 * step + 4 * c < p.r;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        br[q][t] = in ? __ldg(reinterpret_cast<const uint2*>(b0 + ((long long)ad * p.N + 2 * t) * p.r + 16 * step))
                      : make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * i + 8 * e + g;
          v[q][i][e] = make_uint2(0u, 0u);
          if ((rows >> row) & 1u)
            v[q][i][e] = *reinterpret_cast<const uint2*>(p.v + (long long)(row0 + row) * p.rp + 16 * step + 4 * c);
        }
      if (on && ++step == steps) {
        step = 0;
        for (int d = 0; d < p.groups; ++d) {
          ++pass;
          left &= left - 1;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t)
          mma16816(acc[i][t], v[q][i][0].x, v[q][i][1].x, v[q][i][0].y, v[q][i][1].y, br[q][t].x, br[q][t].y);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!mine[i][e]) continue;
      uint32_t* yw = reinterpret_cast<uint32_t*>(&y[i][e]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&yw[t]));
        const __half2 h = __floats2half2_rn(fmaf(acc[i][t][2 * e], unit[i][e], f.x),
                                            fmaf(acc[i][t][2 * e + 1], unit[i][e], f.y));
        yw[t] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.y + (long long)(row0 + 16 * i + 8 * e + g) * p.N + n0 + 8 * c) = y[i][e];
    }
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, int threads, int cluster, const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = cluster;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Blocks of 32 rows from 128 rows on: enough blocks to fill the card, and each
// adapter operand is used for twice as many rows (where the registers hold the
// sums of 32 rows, in the first product).
int row_tiles(int M) { return M >= 128 ? 2 : 1; }
int down_tiles(int M, int r) { return r <= 64 ? row_tiles(M) : 1; }

}  // namespace

void lora_plan(LoraParams* p, int sms) {
  const int rows = 16 * down_tiles(p->M, p->r), blocks = (p->M + rows - 1) / rows;
  int most = p->M < rows ? p->M : rows;  // different adapters in a block
  if (p->adapters < most) most = p->adapters;
  p->rp = (p->r + 15) / 16 * 16;
  p->passes = p->M >= 128 ? 1 : most;
  p->groups = p->M >= 128 ? 1 : (most + 3) / 4;
  // clusters of up to 8 CTAs, while there are few CTAs and a step for every warp
  int s = 1;
  while (s < 8 && 2 * s * blocks * p->passes <= 4 * sms && p->K / 32 >= 2 * s * kDownWarps) s *= 2;
  p->splits = s;
}

cudaError_t launch_lora_down(const LoraParams& p, cudaStream_t stream) {
  const int nt = p.r <= 8 ? 1 : p.r <= 16 ? 2 : p.r <= 32 ? 4 : p.r <= 64 ? 8 : 16;
  const int mt = down_tiles(p.M, p.r);
  const dim3 grid((p.M + 16 * mt - 1) / (16 * mt), p.splits, p.passes);
#define W4A16_DOWN(MT, NT) \
  if (mt == MT && nt == NT) return launch(lora_down_kernel<MT, NT>, grid, kDownWarps * 32, p.splits, p, stream);
  W4A16_DOWN(1, 1) W4A16_DOWN(1, 2) W4A16_DOWN(1, 4) W4A16_DOWN(1, 8) W4A16_DOWN(1, 16)
  W4A16_DOWN(2, 1) W4A16_DOWN(2, 2) W4A16_DOWN(2, 4) W4A16_DOWN(2, 8)
#undef W4A16_DOWN
  return cudaErrorInvalidValue;
}

cudaError_t launch_lora_up(const LoraParams& p, cudaStream_t stream) {
  const int mt = row_tiles(p.M), blocks = (p.M + 16 * mt - 1) / (16 * mt);
  const dim3 grid(blocks, p.N / (kUpWarps * 32), p.groups);
  return mt == 1 ? launch(lora_up_kernel<1>, grid, kUpWarps * 32, 1, p, stream)
                 : launch(lora_up_kernel<2>, grid, kUpWarps * 32, 1, p, stream);
}

}  // namespace w4a16
