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
enum KvSite {
  kKvSiteQStart = 101, kKvSiteLen = 102, kKvSitePage = 103, kKvSiteAdapter = 104, kKvSitePosition = 105, kKvSiteTree = 106,
  kKvSiteIndex = 107
};

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

// The request that owns row t of the new tokens (by its starts: the last one that does not begin after it).
__device__ __forceinline__ int kv_owner(const KvParams& p, int t) {
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same by a warp, for one row: 32 starts at a time.
__device__ __forceinline__ int kv_owner_by_warp(const KvParams& p, int t) {
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + ((int)(threadIdx.x & 31) + 1) * step;
    const int n = __popc(__ballot_sync(0xffffffffu, at < hi && p.q_start[at] <= t));
    lo = min(lo + n * step, hi - 1);
    hi = min(hi, lo + step);
  }
  return lo;
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
  const int* tree;          // for trees: int32 [T][tree_words], bit j of a row: it sees its request's j-th new token
  int tree_words;
};

// Trees: a row sees all cached tokens before the new ones (the last `window` up to its position, which is the last of
// those plus the new tokens that it sees), and the new ones whose bits are set.

// A row's first visible token among those before the new ones, the first new token where it sees none of them.
__device__ __forceinline__ int kv_tree_lo(const KvAttnParams& p, const KvSeq& s, int i) {
  const int first = s.len - s.nq;
  if (p.window <= 0) return 0;
  const int* row = p.tree + (long long)(s.q0 + i) * p.tree_words;
  int seen = 0;
  for (int w = 0; w < p.tree_words && w * 32 < s.nq; ++w) {
    const int left = s.nq - w * 32;
    seen += __popc((uint32_t)row[w] & (left < 32 ? (1u << left) - 1u : ~0u));
  }
  return min(max(first + seen - p.window, 0), first);
}

// Which of the tokens t0 .. t0 + 31 row i of a request sees; lo as above.
__device__ __forceinline__ uint32_t kv_tree_see(const KvAttnParams& p, const KvSeq& s, int i, int lo, int t0) {
  const int j0 = t0 - (s.len - s.nq);  // the first of them among the new tokens; all before these count as set bits
  const int w = j0 >> 5;
  const int* row = p.tree + (long long)(s.q0 + i) * p.tree_words;
  const uint32_t a = w < 0 ? ~0u : w < p.tree_words ? (uint32_t)row[w] : 0u;
  const uint32_t b = w + 1 < 0 ? ~0u : w + 1 < p.tree_words ? (uint32_t)row[w + 1] : 0u;
  uint32_t see = __funnelshift_r(a, b, (uint32_t)j0);
  const int left = s.nq - j0, hidden = lo - t0;
  if (left < 32) see &= left <= 0 ? 0u : (1u << left) - 1u;
  if (hidden > 0) see &= hidden >= 32 ? 0u : ~0u << hidden;
  return see;
}

// A row's sum of probabilities, infinite for a row that sees no token, so that its result is zero.  One that sees some
// and whose scores are all minus infinity has a sum of 0, too: its softmax is not defined, and the result NaN.
// (The look at the bits is not inlined: hardly ever made, its code at every row's end made short trees 10% slower.)
__device__ __noinline__ static bool kv_tree_sees(const int* row, int words, int nq, int len, int window) {
  const int first = len - nq;
  int seen = 0, there = 0;  // bits of new tokens, and of those at positions from 0 on
  for (int j = 0; j < nq && j < 32 * words; ++j) {
    const int bit = ((uint32_t)row[j >> 5] >> (j & 31)) & 1u;
    seen += bit;
    if (first + j >= 0) there += bit;
  }
  return there > 0 || (window > 0 ? min(max(first + seen - window, 0), first) : 0) < first;
}
__device__ __forceinline__ float kv_tree_sum(const KvAttnParams& p, const KvSeq& s, int i, float sum) {
  const bool empty = sum == 0.f && !kv_tree_sees(p.tree + (long long)(s.q0 + i) * p.tree_words, p.tree_words, s.nq, s.len, p.window);
  return empty ? __builtin_huge_valf() : sum;
}

// row / group, exact for 32-bit rows.
__device__ __forceinline__ int kv_div_group(const KvAttnParams& p, int row) {
  return p.group_magic ? (int)__umul64hi((unsigned long long)(uint32_t)row, p.group_magic) : row;
}

cudaError_t launch_kv_append(const KvParams& p, int D, const uint16_t* k, const uint16_t* v, const long long (&st)[4],
                             cudaStream_t stream);
cudaError_t launch_kv_read(const KvParams& p, int D, uint16_t* k, uint16_t* v, const long long (&st)[4],
                           cudaStream_t stream);
// nb: blocks of 8 query rows that share a pass over the cache (1 or 2).  Where p.tree is set the new
// tokens see each other as its bits say, else causally; of the prompt kernel too.
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

// ---- rotary positions and append (kv_cache.cu) ----
constexpr int kRopeAxes = 4;
struct KvRopeParams {
  KvParams kv;
  const uint16_t *q, *k, *v;  // fp16 [T][heads or hkv][D] with strides
  uint16_t* q_out;
  long long q_ts, q_hs, o_ts, o_hs, k_ts, k_hs, v_ts, v_hs;  // elements
  int heads;
  long long warps;            // that share the work (filled in by launch_kv_rope_append)
  const int* positions;       // [axes][T]
  const float* table;         // [table_rows][rot / 2] of (cos, sin)
  int axes, table_rows, rot;
  int grouped;                // the pairs of every D / 32 consecutive ones share an axis
  unsigned long long axis[2];  // two bits a pair
};
cudaError_t launch_kv_rope_append(const KvRopeParams& p, int D, bool interleaved, int sms, cudaStream_t stream);

// ---- trees, compaction, page copies (kv_tree.cu, kv_move.cu) ----
cudaError_t launch_kv_tree(const KvParams& p, const int* parents, int words, int* mask, int* positions, cudaStream_t stream);
constexpr int kMoveCaches = 128;  // of a launch
struct KvCaches {
  uint8_t* at[kMoveCaches];
};
struct KvCompactParams {
  KvParams kv;          // its cache is not used
  int caches;
  const int* into;      // [B][into_pages], the kept tokens' pages; nullptr: where they are
  int into_pages;
  const int *index, *kept;
  int* new_lens;        // nullptr where another launch writes them
  int max_q;
  int look;             // into: every CTA looks at its request's indexes (filled in by launch_kv_compact)
};
cudaError_t launch_kv_compact(const KvCompactParams& p, const KvCaches& c, int D, int sms, cudaStream_t stream);
cudaError_t launch_kv_copy_pages(const KvCaches& c, int caches, int n_pages, long long page_bytes, const int* src,
                                 const int* dst, int pairs, int* status, cudaStream_t stream);
// Warps of a CTA at most, and floats of a part in the workspace at most (16 rows).
constexpr int kKvAttnWarps = 8;
constexpr int kv_attn_part_floats(int D) { return 16 * (D + 4 + 2); }

}  // namespace w4a16
