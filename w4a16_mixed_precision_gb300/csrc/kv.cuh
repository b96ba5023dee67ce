// kv.cuh -- the 4-bit paged key/value cache: its layout, the arguments its
// kernels share, and how they find a token's place in it.
//
// A vector x (one token, one head, D channels of a key or a value) is held as
// D 4-bit codes c and two fp16 numbers: x ~ s * (c - 8) + o with
// s = (max - min) / 15 and o = min + 8 s.  One scale for the whole vector
// means that the scale and the offset leave both products of attention: with
// z = o - 8 s,
//     q . k = s (q . c) + z sum(q),    sum_t p_t v_t = sum_t (p_t s_t) c_t + sum_t p_t z_t,
// so the tensor cores multiply the codes themselves and no per-element
// dequantisation is left.
//
// The unit of the layout is a granule: 16 consecutive tokens of one head,
//     [K codes 16 * D/2 | V codes 16 * D/2 | 16 x (ks, ko, vs, vo) fp16]
// = 16 (D + 8) bytes, one bulk copy.  A page holds page_size / 16 granules of
// every head, head-major; the cache is n_pages such pages.
//   K codes: token-major, channel i of a token at nibble i of its D/2 bytes.
//     Lane (g, c) of a warp reads D/4 channels of tokens g and g + 8 with one
//     shared load each; as the A operand of a 16-token MMA they need no
//     permutation because the query is loaded in the same channel order.
//   V codes: the contraction runs over tokens, so an operand register holds
//     one channel of two tokens.  32-bit words pair the tokens 2c, 2c + 1
//     (low and high half) of four channels: word w of lane (g, c) in half hf
//     (tokens 8 hf + 2c, + 1) holds channels g D/8 + 4w .. + 3, at
//     hf * 4D + (4 g + c) * D/8 + 4 w bytes.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace w4a16 {

constexpr int kGranule = 16;  // tokens
__host__ __device__ constexpr int kv_granule_bytes(int D) { return kGranule * (D + 8); }

struct KvParams {
  uint8_t* cache;
  long long page_bytes, head_bytes;  // strides of a page and of a head in it
  int n_pages, max_pages;            // pages of the cache; columns of the page table
  int hkv, page, page16;             // key heads; tokens and granules per page
  uint32_t page16_magic;             // ceil(2^32 / page16), 0 for page16 = 1
  int B, T;                          // requests, new tokens of all of them
  const int *table, *lens, *q_start;
  int* status;
};

__device__ __forceinline__ void kv_fail(const KvParams& p, int site) {
  atomicCAS(p.status + 1, 0, site);
  atomicOr(p.status, kStatusBounds);
}

// Sites of failed checks of device-side inputs (the word after the status word).
enum KvSite { kKvSiteQStart = 101, kKvSiteLen = 102, kKvSitePage = 103, kKvSiteAdapter = 104 };

// Brings the lengths, starts and page table towards L2 before the wait for the
// previous kernel (which may still be writing them: a prefetch takes no value).
// thread: index among all threads of the grid, a 128-byte line each.
__device__ __forceinline__ void kv_prefetch_plan(const KvParams& p, long long thread) {
  const long long table = (long long)p.B * p.max_pages;
  const char* at = nullptr;
  if (thread * 32 < table) at = reinterpret_cast<const char*>(p.table) + thread * 128;
  if (at) asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
  if (thread * 32 < p.B) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p.lens) + thread * 128));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p.q_start) + thread * 128));
  }
}

// Page of a granule of a request (g16 / page16) and its place inside the page.
// page16 <= 64 and g16 < 2^26, where the rounded-up reciprocal is exact.
__device__ __forceinline__ int kv_div_page(const KvParams& p, int g16) {
  return p.page16_magic ? (int)__umulhi((uint32_t)g16, p.page16_magic) : g16;
}

// New tokens [q0, q0 + nq) and cached length (with them) of request b; a
// request whose entries contradict each other has no new tokens.
struct KvSeq {
  int q0, nq, len;
};

__device__ __forceinline__ KvSeq kv_seq(const KvParams& p, int b, bool report) {
  KvSeq s;
  s.q0 = p.q_start[b];
  const int q1 = p.q_start[b + 1];
  s.len = p.lens[b];
  s.nq = q1 - s.q0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > p.T) {
    if (report) kv_fail(p, kKvSiteQStart);
    s.q0 = s.nq = 0;
  }
  const long long cap = (long long)p.max_pages * p.page;
  if (s.len < 0 || s.len > cap) {
    if (report) kv_fail(p, kKvSiteLen);
    s.len = s.len < 0 ? 0 : (int)cap;
    s.nq = 0;
  }
  return s;
}

struct KvAttnParams {
  KvParams kv;
  const uint16_t* q;        // fp16 [T][heads][D] with strides
  long long q_ts, q_hs;     // elements
  uint16_t* out;            // fp16 [T][heads][D]
  int heads, group;         // query heads, and of them per key head
  int stripes;              // CTAs that share all items of the prompt kernel where these are cut
  unsigned long long group_magic;  // ceil(2^64 / group), 0 for group = 1
  int window;               // > 0: a query sees that many positions, its own included
  float scale_log2;         // softmax scale * log2(e)
  int whole_blocks;         // pages hold whole blocks: one copy each
  int min_rows;             // requests with up to so many query rows per key head are left to another launch
  int max_rows;             // requests with more query rows per key head are left to another launch
  int* counters;            // [grid], zero between calls
  float* partials;          // [2 grid] parts of segments cut between CTAs, kv_attn_part_floats(D) at most
  float* firsts;            // [grid][warps] parts that a warp leaves before its stripe is done
  unsigned long long timeout_ns;
};

// row / group, exact for 32-bit rows.
__device__ __forceinline__ int kv_div_group(const KvAttnParams& p, int row) {
  return p.group_magic ? (int)__umul64hi((unsigned long long)(uint32_t)row, p.group_magic) : row;
}

cudaError_t launch_kv_append(const KvParams& p, int D, const uint16_t* k, const uint16_t* v, const long long (&st)[4],
                             cudaStream_t stream);
cudaError_t launch_kv_read(const KvParams& p, int D, uint16_t* k, uint16_t* v, const long long (&st)[4],
                           cudaStream_t stream);
// nb: blocks of 8 query rows that share a pass over the cache (1 or 2)
cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int nb, int grid, cudaStream_t stream);
cudaError_t kv_attn_set_smem_limit();
cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, int grid, cudaStream_t stream);
// Items (256 rows of a request and key head) at most: one part-filled for each request.
constexpr long long kv_prefill_items(long long tokens, int requests, int hkv, int group) {
  return (tokens * group / 256 + requests) * hkv;
}
// Floats of a part of an item (256 rows) that stripes cut; two for every CTA.
constexpr int kv_prefill_part_floats(int D) { return 256 * (D + 4); }
cudaError_t kv_prefill_set_smem_limit();
// Warps of a CTA at most, and floats of a part in the workspace at most (16 rows).
constexpr int kKvAttnWarps = 8;
constexpr int kv_attn_part_floats(int D) { return 16 * (D + 4 + 2); }

}  // namespace w4a16
