// lora.cu -- low-rank adapters of many requests beside a shared product:
//     y[m] += scaling[a] * (x[m] . A[a]^T) . B[a]^T,   a = index[m] (none if negative),
// A[a] r x K and B[a] N x r in fp16.  Up to a few hundred rows one kernel after the
// product, v = scaling x . A^T staying in shared memory between its two halves; for
// more rows two, so that the second can take 128 rows at a time.
//
// Bound: for few rows reading the adapters in use, r (K + N) fp16 each; for
// many rows reading x, and reading and writing y.
//   * Few rows: an item is up to 16 rows of one adapter, in any places, found in the
//     kernel; a cluster takes an item, so that every adapter in use is read once for
//     16 rows of it.  Many rows: these are taken in blocks, and a block makes one
//     pass for each different adapter among its rows (one, for the rows of a prompt),
//     with the other rows masked.  So any order of rows is right in both.
//   * mma.sync with the rows as the 16-row operand.  The k order is permuted
//     alike in both operands so that every lane loads 16 consecutive bytes.
//   * First product: K is split over the warps of a CTA and the CTAs of a
//     cluster; all parts are summed through distributed shared memory, in the
//     same order.  Second product, few rows: the cluster's warps split the N
//     columns, with the operands of the next four groups of columns in flight.
//     Many rows: a warp keeps its operand columns in registers and passes over
//     the block's rows.
//   * v is normalised by a power of two per row (so that no magnitude of x leaves
//     fp16's range) and rounded to fp16 for the second product: one rounding of
//     2^-12 per term of a sum that is itself an addition to y.
//
// Measured beside the product (its own time first), 4096 x 12288: 32 rows of 21
// adapters of rank 16 13.9 + 9.3 us; 48 of 21, rank 64 (44 MB) 15.7 + 14, 3.2 TB/s; of
// rank 128 15.7 + 28, 3.1 TB/s; one row, 4096 x 4096, rank 16, 5.9 + 5.2; 2000 rows of
// prompts 162 + 43 (15 of them reading and writing y, 3 leaving the workspace zero).  A single row's time is three
// trips to memory (index, A and x, B) and a barrier of the cluster.
#include "lora.h"

#include <cuda_fp16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace w4a16 {

namespace {

constexpr int kWarps = 8;
constexpr int kFewRows = 512;  // room of the kernel that does both products: 320 rows at most, two for each thread
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// y (eight columns of a row, loaded before) + u * acc, rounded, to its place.
// e: the row of the tile's pair (g or g + 8).
__device__ __forceinline__ void add_row(uint16_t* at, uint4 y, const float (&acc)[4][4], int e, float u) {
  uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&yw[t]));
    const __half2 h = __floats2half2_rn(fmaf(acc[t][2 * e], u, f.x), fmaf(acc[t][2 * e + 1], u, f.y));
    yw[t] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(at) = y;
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

// v and unit of blocks of rows, for the workspace.  MT: 16-row tiles per block; NT:
// 8-rank tiles (r <= 8 NT).  Grid: blocks of rows; CTAs of the cluster (parts of K).
template <int MT, int NT>
__global__ void __launch_bounds__(kWarps * 32, NT <= 8 ? 2 : 1) lora_down_kernel(const LoraParams p) {
  constexpr int kRows = 16 * MT, kRanks = 8 * NT, kRp = (kRanks + 15) / 16 * 16, kAcc = MT * NT * 4;
  // half of the warps leave their sums to the other half, three times; then the CTA's sum
  __shared__ float red[kWarps / 2][kAcc][32];
  __shared__ float total[kRows][kRanks + 1];
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * kRows, rank = blockIdx.y;
  const Block k = block_adapters(p, row0, kRows);
  const int count = __popc(k.leaders);
  // ---- x . A^T: this warp's 32-wide K steps --------------------------------------------
  {
    const int steps = p.K / 32, parts = p.splits * kWarps, part = rank * kWarps + warp;
    const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
    float acc[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
    uint32_t left = k.leaders;
    for (int q = 0; q < count; ++q, left &= left - 1) {
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
    // the sum over the warps, in a fixed order
#pragma unroll
    for (int half = kWarps / 2; half >= 1; half >>= 1) {
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
  }
  if (p.splits > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // ---- v: the sum over the cluster, scaled, normalised, fp16; each CTA a share of the rows ----
  for (int row = rank * kWarps + warp; row < kRows; row += kWarps * p.splits) {
    const int ad = __shfl_sync(0xffffffffu, k.mine, row);
    const bool on = ad >= 0;
    const float scaling = on ? p.scaling[ad] : 0.f;
    float s[(kRp + 31) / 32], top = 0.f;
#pragma unroll
    for (int i = 0; i < (kRp + 31) / 32; ++i) {
      const int j = 32 * i + lane;
      s[i] = 0.f;
      if (on && j < p.r) {
        if (p.splits == 1) {
          s[i] = total[row][j];
        } else {
          float part[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) part[q] = q < p.splits ? ld_cluster(smem_addr(&total[row][j]), (uint32_t)q) : 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q) s[i] += part[q];
        }
        s[i] *= scaling;
      }
      top = fmaxf(top, fabsf(s[i]));
    }
#pragma unroll
    for (int q = 1; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
    // 2^exponent of the row's largest magnitude
    const float u = top > 1e-30f ? __uint_as_float(__float_as_uint(top) & 0x7F800000u) : 1.f;
#pragma unroll
    for (int i = 0; i < (kRp + 31) / 32; ++i)
      if (on && 32 * i + lane < p.rp)
        p.v[(long long)(row0 + row) * p.rp + 32 * i + lane] = __half_as_ushort(__float2half_rn(s[i] / u));
    if (lane == 0 && on) p.unit[row0 + row] = u;
  }
  if (p.splits > 1) {  // nobody reads this CTA's shared memory any more
    cluster_arrive();
    cluster_wait();
  }
}

// Both products for few rows.  An item is up to 16 rows of one adapter, in any
// places; a cluster takes an item (or the items z, z + gridDim.z, ...), so that every
// adapter in use is read once.  Where there are fewer items than clusters, several
// clusters share one: each sums the whole first product, and takes a share of the
// columns of the second.  NT: 8-rank tiles (r <= 8 NT).  Grid: CTAs of the cluster
// (parts of K, then of N); clusters.
template <int NT>
__global__ void __launch_bounds__(kWarps * 32, NT <= 2 ? 2 : 1) lora_few_kernel(const LoraParams p) {
  constexpr int kRanks = 8 * NT, kRp = (kRanks + 15) / 16 * 16, kAcc = NT * 4;
  // half of the warps leave their sums to the other half, three times; then the CTA's sum
  __shared__ float red[kWarps / 2][kAcc][32];
  __shared__ float total[16][kRanks + 1];
  __shared__ __align__(16) __half v[16][kRp + 8];
  __shared__ float unit[16];
  __shared__ __align__(16) int adapter[kFewRows];        // of each row, -1 for none
  __shared__ int starts[kFewRows / 32];                  // items that begin in each 32 rows
  __shared__ int item_rows[16], item_ad, item_at;
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int rank = blockIdx.y;

  // ---- the items: a row begins one if 16 n rows before it have its adapter -----------------
  // this thread's rows, tid + 256 i: their adapters, places among those ones' rows, and the
  // items they begin
  constexpr int kMine = kFewRows / (kWarps * 32);
  int mine[kMine], at[kMine], item_of[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int row = tid + kWarps * 32 * i;
    mine[i] = row < p.M ? p.index[row] : -1;
    if (mine[i] >= p.adapters) {
      atomicCAS(p.status + 1, 0, kLoraSite);
      atomicOr(p.status, kStatusBounds);
      mine[i] = -1;
    }
    if (mine[i] < 0) mine[i] = -1;
    adapter[row] = mine[i];
    at[i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int row = tid + kWarps * 32 * i, word = i * kWarps + warp;
    item_of[i] = -1;
    if (32 * word >= p.M) continue;  // alike in the warp
    for (int j = 0; j <= 8 * word + 7 && 4 * j < p.M; ++j) {  // up to the warp's last row
      const int4 q = reinterpret_cast<const int4*>(adapter)[j];
      at[i] += (q.x == mine[i] && 4 * j < row) + (q.y == mine[i] && 4 * j + 1 < row) +
               (q.z == mine[i] && 4 * j + 2 < row) + (q.w == mine[i] && 4 * j + 3 < row);
    }
    const bool begin = mine[i] >= 0 && at[i] % 16 == 0;
    const uint32_t begins = __ballot_sync(0xffffffffu, begin);
    if (begin) item_of[i] = __popc(begins & ((1u << lane) - 1));
    if (lane == 0) starts[word] = __popc(begins);
  }
  __syncthreads();
  int items = 0;
  for (int w = 0; 32 * w < p.M; ++w) {
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (item_of[i] >= 0 && w < i * kWarps + warp) item_of[i] += starts[w];
    items += starts[w];
  }
  if (items == 0) return;
  const int clusters = gridDim.z, z = blockIdx.z;
  const int shares = items <= clusters ? min(clusters / items, p.shares) : 1;
  const int share = items <= clusters ? z / items : 0;
  if (share >= shares) return;  // alike in all CTAs of the cluster

  for (int item = items <= clusters ? z % items : z; item < items; item += clusters) {
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (item_of[i] == item) {
        item_ad = mine[i];
        item_at = at[i];
      }
    if (tid < 16) item_rows[tid] = -1;
    __syncthreads();
    const int ad = item_ad;
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (mine[i] == ad && at[i] >= item_at && at[i] < item_at + 16) item_rows[at[i] - item_at] = tid + kWarps * 32 * i;
    __syncthreads();
    const int row0 = item_rows[g], row1 = item_rows[g + 8];  // of this lane, -1 where there is none

    // ---- x . A^T: this warp's 32-wide K steps ------------------------------------------
    {
      const int steps = p.K / 32, parts = p.splits * kWarps, part = rank * kWarps + warp;
      const int s0 = steps * part / parts, s1 = steps * (part + 1) / parts;
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
      const uint16_t* a = p.a + (long long)ad * p.r * p.K + c * 8;
      const uint16_t* x0 = p.x + (long long)row0 * p.K + c * 8;
      const uint16_t* x1 = p.x + (long long)row1 * p.K + c * 8;
      constexpr int kTogether = NT <= 4 ? 4 : NT <= 8 ? 2 : 1;  // steps whose loads go out together
#pragma unroll kTogether
      for (int s = s0; s < s1; ++s) {
        uint4 xr[2], ar[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          ar[j] = j * 8 + g < p.r ? __ldg(reinterpret_cast<const uint4*>(a + (long long)(j * 8 + g) * p.K + s * 32))
                                  : make_uint4(0u, 0u, 0u, 0u);
        xr[0] = row0 >= 0 ? *reinterpret_cast<const uint4*>(x0 + s * 32) : make_uint4(0u, 0u, 0u, 0u);
        xr[1] = row1 >= 0 ? *reinterpret_cast<const uint4*>(x1 + s * 32) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma16816(acc[j], xr[0].x, xr[1].x, xr[0].y, xr[1].y, ar[j].x, ar[j].y);
          mma16816(acc[j], xr[0].z, xr[1].z, xr[0].w, xr[1].w, ar[j].z, ar[j].w);
        }
      }
      // the sum over the warps, in a fixed order
#pragma unroll
      for (int half = kWarps / 2; half >= 1; half >>= 1) {
        if (warp >= half && warp < 2 * half) {
#pragma unroll
          for (int t = 0; t < kAcc; ++t) red[warp - half][t][lane] = acc[t / 4][t % 4];
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
          for (int t = 0; t < kAcc; ++t) acc[t / 4][t % 4] += red[warp][t][lane];
        }
        __syncthreads();
      }
      if (warp == 0) {
#pragma unroll
        for (int t = 0; t < kAcc; ++t) {
          const int j = t / 4, e = t % 4;
          total[g + 8 * (e >> 1)][8 * j + 2 * c + (e & 1)] = acc[j][e];
        }
      }
    }
    if (p.splits > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // ---- v: the sum over the cluster, scaled, normalised, fp16; every CTA for itself -----------
    const float scaling = p.scaling[ad];
    for (int row = warp; row < 16; row += kWarps) {
      const bool on = item_rows[row] >= 0;
      float s[(kRp + 31) / 32], top = 0.f;
#pragma unroll
      for (int i = 0; i < (kRp + 31) / 32; ++i) {
        const int j = 32 * i + lane;
        s[i] = 0.f;
        if (on && j < p.r) {
          if (p.splits == 1) {
            s[i] = total[row][j];
          } else {
            float part[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              part[q] = q < p.splits ? ld_cluster(smem_addr(&total[row][j]), (uint32_t)q) : 0.f;
#pragma unroll
            for (int q = 0; q < 8; ++q) s[i] += part[q];
          }
          s[i] *= scaling;
        }
        top = fmaxf(top, fabsf(s[i]));
      }
#pragma unroll
      for (int q = 1; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
      // 2^exponent of the row's largest magnitude
      const float u = top > 1e-30f ? __uint_as_float(__float_as_uint(top) & 0x7F800000u) : 1.f;
#pragma unroll
      for (int i = 0; i < (kRp + 31) / 32; ++i)
        if (32 * i + lane < kRp) v[row][32 * i + lane] = __float2half_rn(s[i] / u);
      if (lane == 0) unit[row] = u;
    }
    if (p.splits > 1) cluster_arrive();  // this CTA has read the others' sums
    __syncthreads();

    // ---- y += v . B^T: this warp's groups of 32 columns ------------------------------------
    constexpr int kAhead = 4;                  // (group, step) pairs whose loads are in flight
    constexpr int kRanksStep = NT >= 4 ? 32 : 16, kHalves = kRanksStep / 16;  // ranks of a step: 8 or 16 bytes a lane
    const int groups = p.N / 32, parts = shares * p.splits * kWarps, part = (share * p.splits + rank) * kWarps + warp;
    const int n_first = groups * part / parts, n_last = groups * (part + 1) / parts;
    const int steps = (p.r + kRanksStep - 1) / kRanksStep;
    // operand column g of tile t is output column 8 (g / 2) + 2 t + g % 2 of the
    // group's 32, so that a lane's results are 8 consecutive columns of y
    const uint16_t* b = p.b + ((long long)ad * p.N + 8 * (g >> 1) + (g & 1)) * p.r + 4 * kHalves * c;
    uint16_t* const y_at[2] = {p.y + (long long)row0 * p.N + 8 * c, p.y + (long long)row1 * p.N + 8 * c};
    const bool on[2] = {row0 >= 0, row1 >= 0};
    uint32_t br[kAhead][4][2 * kHalves];
    uint4 y[kAhead][2];  // with a group's last step: its rows g and g + 8
    int load_n = n_first, load_step = 0;
    auto load = [&](uint32_t(&bq)[4][2 * kHalves], uint4(&yq)[2]) {
      if (load_n >= n_last) return;
      const bool in = kRanksStep * load_step + 4 * kHalves * c < p.r;
      const uint16_t* src = b + (long long)(32 * load_n) * p.r + kRanksStep * load_step;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        if constexpr (kHalves == 2) {
          const uint4 q = in ? __ldg(reinterpret_cast<const uint4*>(src + 2 * t * p.r)) : make_uint4(0u, 0u, 0u, 0u);
          bq[t][0] = q.x; bq[t][1] = q.y; bq[t][2] = q.z; bq[t][3] = q.w;
        } else {
          const uint2 q = in ? __ldg(reinterpret_cast<const uint2*>(src + 2 * t * p.r)) : make_uint2(0u, 0u);
          bq[t][0] = q.x; bq[t][1] = q.y;
        }
      }
      if (++load_step < steps) return;
      load_step = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (on[e]) yq[e] = *reinterpret_cast<const uint4*>(y_at[e] + 32 * load_n);
      ++load_n;
    };
#pragma unroll
    for (int q = 0; q < kAhead; ++q) load(br[q], y[q]);
    int n = n_first, step = 0;
    float acc[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    while (n < n_last) {
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        if (n < n_last) {  // uniform
#pragma unroll
          for (int d = 0; d < kHalves; ++d) {
            const int at_rank = kRanksStep * step + 4 * kHalves * c + 4 * d;
            const uint2 v0 = *reinterpret_cast<const uint2*>(&v[g][at_rank]);
            const uint2 v1 = *reinterpret_cast<const uint2*>(&v[g + 8][at_rank]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
              mma16816(acc[t], v0.x, v1.x, v0.y, v1.y, br[q][t][2 * d], br[q][t][2 * d + 1]);
          }
          if (++step == steps) {
            step = 0;
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (on[e]) add_row(y_at[e] + 32 * n, y[q][e], acc, e, unit[8 * e + g]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
            ++n;
          }
          load(br[q], y[q]);
        }
      }
    }
    if (p.splits > 1) cluster_wait();  // nobody reads this CTA's sums any more
    __syncthreads();                   // nor its v, its rows
  }
}

// y += v . B^T for blocks of 128 rows: a warp keeps 32 columns of B in registers
// (a step of 16 ranks at a time beyond 64) and passes over the rows.  ST: steps
// of 16 ranks (r <= 16 ST).  v and unit lie where the product's partial tiles are
// when the workspace serves another call, and those have to be zero between calls:
// the last warp of a block of rows to finish zeroes what the block has read.
template <int ST>
__global__ void __launch_bounds__(kWarps * 32, ST <= 4 ? 2 : 1) lora_up_kernel(const LoraParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * 128, n0 = (blockIdx.y * kWarps + warp) * 32;
  int mine[4];  // the adapters of rows lane, lane + 32, ...
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 32 * i + lane;
    const int ad = row < p.M ? p.index[row] : -1;
    mine[i] = ad < 0 || ad >= p.adapters ? -1 : ad;  // out of range: reported by the first kernel
  }
  const uint16_t* b = p.b + ((long long)n0 + 8 * (g >> 1) + (g & 1)) * p.r + 4 * c;
  while (n0 < p.N) {
    // the next adapter, and its rows
    int ad = -1;
    uint32_t rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t left = __ballot_sync(0xffffffffu, mine[i] >= 0);
      if (ad < 0 && left) ad = __shfl_sync(0xffffffffu, mine[i], __ffs(left) - 1);
    }
    if (ad < 0) break;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rows[i] = __ballot_sync(0xffffffffu, mine[i] == ad);
      if (mine[i] == ad) mine[i] = -1;
    }
    uint2 br[ST][4];
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        br[s][t] = 16 * s + 4 * c < p.r
                       ? __ldg(reinterpret_cast<const uint2*>(b + ((long long)ad * p.N + 2 * t) * p.r + 16 * s))
                       : make_uint2(0u, 0u);
    // tiles of 16 rows, kTogether at a time with their loads in flight
    constexpr int kTogether = ST <= 2 ? 4 : 2;
#pragma unroll 1
    for (int i0 = 0; i0 < 8; i0 += kTogether) {
      uint4 y[kTogether][2];
      uint2 v[kTogether][ST][2];
      float u[kTogether][2];
#pragma unroll
      for (int q = 0; q < kTogether; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tile = i0 + q;
          const uint32_t word = tile < 2 ? rows[0] : tile < 4 ? rows[1] : tile < 6 ? rows[2] : rows[3];
          const bool on = (word >> (16 * (tile & 1) + 8 * e + g)) & 1u;
          const long long row = row0 + 16 * tile + 8 * e + g;
          u[q][e] = 0.f;  // 0 marks a row that is not this adapter's
#pragma unroll
          for (int s = 0; s < ST; ++s) v[q][s][e] = make_uint2(0u, 0u);
          if (on) {
            y[q][e] = *reinterpret_cast<const uint4*>(p.y + row * p.N + n0 + 8 * c);
            u[q][e] = p.unit[row];
#pragma unroll
            for (int s = 0; s < ST; ++s)
              if (16 * s < p.rp) v[q][s][e] = *reinterpret_cast<const uint2*>(p.v + row * p.rp + 16 * s + 4 * c);
          }
        }
#pragma unroll
      for (int q = 0; q < kTogether; ++q) {
        float acc[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            mma16816(acc[t], v[q][s][0].x, v[q][s][1].x, v[q][s][0].y, v[q][s][1].y, br[s][t].x, br[s][t].y);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (u[q][e] != 0.f)
            add_row(p.y + (long long)(row0 + 16 * (i0 + q) + 8 * e + g) * p.N + n0 + 8 * c, y[q][e], acc, e, u[q][e]);
      }
    }
  }
  // release and acquire at the card's scope, for the whole warp by way of its barriers
  int arrived = 0;
  __syncwarp();
  if (lane == 0)
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(arrived) : "l"(p.arrived + blockIdx.x) : "memory");
  if (__shfl_sync(0xffffffffu, arrived, 0) != (int)gridDim.y * kWarps - 1) return;
  __syncwarp();
  if (lane == 0) p.arrived[blockIdx.x] = 0;
  const int rows = min(128, p.M - row0);
  uint4* v = reinterpret_cast<uint4*>(p.v + (long long)row0 * p.rp);
  for (int i = lane; i < rows * p.rp / 8; i += 32) v[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int i = lane; i < rows; i += 32) p.unit[row0 + i] = 0.f;
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, int cluster, const LoraParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
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

}  // namespace

// Few rows, both products in one kernel after marlin_gemm; many, the first product before
// it in the stream (its launch and tail overlap the product's start) and the second after
// it.  Measured with the product, one kernel against two: 128 rows of 21 adapters of rank
// 16 (4096 x 12288) 34 against 98 us, 200 of 2, rank 64, 47 against 56, 276 of 5, rank 64
// (4096 x 4096) 42 against 56; 276 of 3, rank 16, 41 against 38, 400 of 2, rank 64
// (4096 x 12288) 84 against 80.
bool lora_two_kernels(int M, int r) { return M > (r >= 32 ? 320 : 256); }

cudaError_t launch_lora(LoraParams p, int half, int sms, cudaStream_t stream) {
  const int nt = p.r <= 8 ? 1 : p.r <= 16 ? 2 : p.r <= 32 ? 4 : p.r <= 64 ? 8 : 16;
  const int most = p.K / 32 / kWarps < 1 ? 1 : p.K / 32 / kWarps < 8 ? p.K / 32 / kWarps : 8;  // a step for every warp
  if (!lora_two_kernels(p.M, p.r)) {
    // items at most: every adapter in use begins one, and every 16 rows more of it
    const int used = std::min(p.M, p.adapters), items = used + (p.M - used) / 16;
    // clusters of s CTAs that the card holds at a time, where they do not fill its parts: as
    // many as measured (rank 64, 8 rows of 4 adapters beside 4096 x 12288: 14 clusters of 8
    // 18.3 us, 16 of them 23.9; 48 rows of 21 adapters: clusters of 6 29.3 us, of 4 32.6)
    auto clusters = [&](int s) { return std::max(1, (nt <= 2 ? 2 : 1) * (s == 8 ? sms / 10 : sms * 7 / 8 / s)); };
    p.splits = most;
    while (p.splits > 1 && clusters(p.splits) < items) --p.splits;
    p.shares = std::max(1, p.N / 32 / (p.splits * kWarps));
    const long long wanted = (long long)items * p.shares;
    const dim3 grid(1, p.splits, (unsigned)std::min(wanted, (long long)clusters(p.splits)));
    return nt == 1   ? launch(lora_few_kernel<1>, grid, p.splits, p, stream)
           : nt == 2 ? launch(lora_few_kernel<2>, grid, p.splits, p, stream)
           : nt == 4 ? launch(lora_few_kernel<4>, grid, p.splits, p, stream)
           : nt == 8 ? launch(lora_few_kernel<8>, grid, p.splits, p, stream)
                     : launch(lora_few_kernel<16>, grid, p.splits, p, stream);
  }
  if (half == 1) {
    const dim3 grid((p.M + 127) / 128, (p.N / 32 + kWarps - 1) / kWarps);
    return p.r <= 16   ? launch(lora_up_kernel<1>, grid, 1, p, stream)
           : p.r <= 32 ? launch(lora_up_kernel<2>, grid, 1, p, stream)
           : p.r <= 64 ? launch(lora_up_kernel<4>, grid, 1, p, stream)
                       : launch(lora_up_kernel<8>, grid, 1, p, stream);
  }
  const int mt = p.r > 64 ? 1 : 2;  // 32 rows where the registers hold their sums
  const int blocks = (p.M + 16 * mt - 1) / (16 * mt);
  // clusters of up to 8 CTAs, while there is room on the card
  p.splits = 1;
  while (2 * p.splits <= most && 2 * p.splits * blocks <= 2 * sms) p.splits *= 2;
  const dim3 grid(blocks, p.splits);
  return nt == 1   ? launch(lora_down_kernel<2, 1>, grid, p.splits, p, stream)
         : nt == 2 ? launch(lora_down_kernel<2, 2>, grid, p.splits, p, stream)
         : nt == 4 ? launch(lora_down_kernel<2, 4>, grid, p.splits, p, stream)
         : nt == 8 ? launch(lora_down_kernel<2, 8>, grid, p.splits, p, stream)
                   : launch(lora_down_kernel<1, 16>, grid, p.splits, p, stream);
}

}  // namespace w4a16
