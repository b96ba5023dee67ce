// kv_tree.cu -- from the parents of drafted tokens to what each of them sees: bit j of a token's row is
// set where the j-th new token of its request is the token itself or one of its ancestors; its position
// is that of the last cached token before the new ones, and its depth.
//
// A thread follows a token's parents, which come before their children: the bits are met from the highest
// down, so that a word is written once it is left.  Bound: latency, a chain of as many loads as the tree
// is deep; 4 bytes a parent, 4 (words + 1) a row are all there is to move.  A CTA's rows are neighbours, and
// most of their parents among them: it brings those to shared memory first.  Measured: 64 tokens of one request
// 4.3 us, 19,539 of 200 requests (38 levels at most) 8.5 us.
#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr int kTreeThreads = 64, kTreeBack = 192;  // rows of a CTA; rows before them whose parents it brings, too

__global__ void __launch_bounds__(kTreeThreads) kv_tree_kernel(const KvParams p, const int* parents, int words, int* mask,
                                                               int* positions) {
  __shared__ int near_by[kTreeBack + kTreeThreads];
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int t0 = blockIdx.x * kTreeThreads - kTreeBack, t = blockIdx.x * kTreeThreads + threadIdx.x;
  for (int i = threadIdx.x; i < kTreeBack + kTreeThreads; i += kTreeThreads)
    if (t0 + i >= 0 && t0 + i < p.T) near_by[i] = parents[t0 + i];
  // the owner of the warp's first row, and on from there
  const int t_warp = t & ~31;
  KvSeq s{0, 0, 0};
  if (t_warp < p.T) {
    int b = kv_owner_by_warp(p, t_warp);
    if (t < p.T) {
      while (b + 1 < p.B && p.q_start[b + 1] <= t) ++b;
      s = kv_seq(p, b, true);
    }
  }
  __syncthreads();
  if (t < s.q0 || t >= s.q0 + s.nq) return;
  if (s.nq > s.len) kv_fail(p, kKvSiteLen);
  if (s.nq > 32ll * words) kv_fail(p, kKvSiteTree);
  int* row = mask + (long long)t * words;
  int w = words;  // words from here on are written
  uint32_t bits = 0;
  int depth = 0;
  for (int j = t - s.q0; j >= 0;) {
    const int at = s.q0 + j;
    const int up = at >= t0 ? near_by[at - t0] : parents[at];
    ++depth;
    for (; w > (j >> 5); --w) {  // on to a lower word: the one before is whole
      if (w < words) row[w] = (int)bits;
      bits = 0;
    }
    if ((j >> 5) == w) bits |= 1u << (j & 31);
    if (up >= j) {  // not a tree with parents first: the token counts as one without a parent
      kv_fail(p, kKvSiteTree);
      break;
    }
    j = up;
  }
  for (; w >= 0; --w) {
    if (w < words) row[w] = (int)bits;
    bits = 0;
  }
  positions[t] = s.len - s.nq + depth - 1;
}

}  // namespace

cudaError_t launch_kv_tree(const KvParams& p, const int* parents, int words, int* mask, int* positions, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)(((long long)p.T + kTreeThreads - 1) / kTreeThreads));
  cfg.blockDim = dim3(kTreeThreads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_tree_kernel, p, parents, words, mask, positions);
}

}  // namespace w4a16
