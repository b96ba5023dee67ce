// ops_api.cu -- the C ABI of the operators beside the W4A16 product: low-rank
// adapters, and the 4-bit paged key/value cache (argument checks, plans,
// launches).
#include <algorithm>
#include <cmath>
#include <mutex>

#include "kernels.h"
#include "kv.cuh"
#include "lora.h"
#include "marlin.h"

using namespace w4a16;

namespace {

constexpr unsigned long long kTimeoutNs = 2000000000ull;  // 2 s per wait

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

marlin_status_t current_sms(int* sms) {
  int dev;
  if (cudaGetDevice(&dev) != cudaSuccess) return MARLIN_ERR_CUDA;
  return static_cast<marlin_status_t>(device_sms(dev, sms));
}

// ---- adapters ---------------------------------------------------------------------

// The product's workspace, then for many rows v, unit and arrivals.  All of it is zero
// between calls: for another M (or shape) the product's partial tiles lie elsewhere in the
// same buffer, and its reducers take a non-zero word for a sum that has been written.
struct LoraSizes {
  size_t gemm, v_off, unit_off, arrived_off, total;
};

marlin_status_t lora_sizes(int M, int K, int N, int group, int r, int device, LoraSizes* z) {
  const marlin_status_t s = marlin_workspace_bytes(M, K, N, group, device, &z->gemm);
  if (s != MARLIN_OK) return s;
  z->v_off = round_up(z->gemm, 256);
  z->unit_off = z->v_off + round_up((size_t)M * round_up(r, 16) * sizeof(uint16_t), 256);
  z->arrived_off = z->unit_off + round_up((size_t)M * sizeof(float), 256);
  z->total = z->arrived_off + ((size_t)M + 127) / 128 * sizeof(int);
  return MARLIN_OK;
}

// ---- cache -------------------------------------------------------------------------

marlin_status_t check_cache(int n_pages, int hkv, int D, int page) {
  if (n_pages <= 0 || hkv <= 0 || D <= 0 || page <= 0) return MARLIN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MARLIN_ERR_UNSUPPORTED;
  if (page % kGranule != 0 || page > 1024) return MARLIN_ERR_UNSUPPORTED;
  return MARLIN_OK;
}

// Checks what the cache entry points share and fills the kernels' arguments.
marlin_status_t make_kv(KvParams* p, const void* cache, int n_pages, int hkv, int D, int page, const int32_t* table,
                        int max_pages, const int32_t* lens, const int32_t* q_start, int B, int T, void* workspace) {
  if (const marlin_status_t c = check_cache(n_pages, hkv, D, page)) return c;
  if (B < 0 || T < 0 || max_pages <= 0) return MARLIN_ERR_INVALID_ARG;
  // positions are 32-bit; a granule's index must stay below 2^26
  if ((long long)max_pages * page > (1ll << 30)) return MARLIN_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return MARLIN_OK;
  if (!cache || !table || !lens || !q_start || !workspace) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(workspace, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(q_start, 4))
    return MARLIN_ERR_MISALIGNED;
  p->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p->page16 = page / kGranule;
  p->page16_magic = p->page16 == 1 ? 0u : (uint32_t)(((1ull << 32) + p->page16 - 1) / p->page16);
  p->head_bytes = (long long)p->page16 * kv_granule_bytes(D);
  p->page_bytes = p->head_bytes * hkv;
  p->n_pages = n_pages;
  p->max_pages = max_pages;
  p->hkv = hkv;
  p->page = page;
  p->B = B;
  p->T = T;
  p->table = table;
  p->lens = lens;
  p->q_start = q_start;
  p->status = static_cast<int*>(workspace);
  return MARLIN_OK;
}

// Strides of a [T][heads][D] tensor in elements: rows must not overlap backwards
// and every vector must start on an aligned address.
bool strides_ok(long long ts, long long hs, int align) {
  return ts >= 0 && hs >= 0 && ts % align == 0 && hs % align == 0;
}

// Whether no two of T x H rows of D elements share any, tokens or heads outermost.
bool rows_apart(long long ts, long long hs, int T, int H, int D) {
  const auto inside = [D](long long inner, int n, long long outer, int m) {  // n inner rows between two outer ones
    return (n == 1 || inner >= D) && (m == 1 || (outer >= D && (n == 1 || (outer - D) / (n - 1) >= inner)));
  };
  return inside(hs, H, ts, T) || inside(ts, T, hs, H);
}

marlin_status_t kv_copy(bool append, uint16_t* k, int64_t k_ts, int64_t k_hs, uint16_t* v, int64_t v_ts, int64_t v_hs,
                        const void* cache, int n_pages, int hkv, int D, int page, const int32_t* table, int max_pages,
                        const int32_t* lens, const int32_t* q_start, int B, int T, void* workspace,
                        marlin_stream_t stream) {
  KvParams p{};
  const marlin_status_t s =
      make_kv(&p, cache, n_pages, hkv, D, page, table, max_pages, lens, q_start, B, T, workspace);
  if (s != MARLIN_OK || B == 0 || T == 0) return s;
  if (!k || !v) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !strides_ok(k_ts, k_hs, 8) || !strides_ok(v_ts, v_hs, 8))
    return MARLIN_ERR_MISALIGNED;
  const long long st[4] = {k_ts, k_hs, v_ts, v_hs};
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = append ? launch_kv_append(p, D, k, v, st, cs) : launch_kv_read(p, D, k, v, st, cs);
  return e == cudaSuccess ? MARLIN_OK : MARLIN_ERR_CUDA;
}

// ---- attention ----------------------------------------------------------------------

// More query rows per key head than this go to the tcgen05 kernel.  Measured with 128
// channels, streaming kernel against tcgen05, by the rows: 8 requests of 8000 tokens, 64 heads
// on 8, 48 rows 79 against 105 us, 64 99 / 105, 80 119 / 105; one of 32,000, 32 heads on 32,
// 48 138 / 176, 64 175 / 175, 80 216 / 176; 32 of 2000, 48 87 / 86, 64 109 / 86; 64 channels, 8
// of 4000, 80 51 / 59, 96 59 / 59, 128 75 / 59.  Few items are the exception, whatever the
// rows: one request of 1000, 64 heads on 8, 160 rows 16 / 32, of 8000 43 / 126 (an item that
// many stripes cut is joined part by part).
// Trees have the same bound, although their parts, which a second kernel joins, would allow 48: it is also where a
// probability times its value's scale goes from two fp16 numbers to one.  Streaming against tcgen05: 8 requests of 8000
// tokens, 64 heads on 8, 32 rows 50 against 63 us, 64 80 / 65; 32 of 2000, 32 58 / 78, 64 89 / 77; one of 8000, 32
// 26 / 25, 64 30 / 26; one of 100,000, 32 86 / 113, 64 149 / 117; 64 channels, 8 of 4000, 32 25 / 35, 64 36 / 37.
constexpr int kPrefillRows = 64;

struct AttnPlan {
  int grid, nb;
  size_t counters_off, partials_off, firsts_off, prompt_off, bytes;
};

// [status 256 B][arrivals of both kernels][parts of the streaming kernel][parts of the
// tcgen05 kernel, where a request can have enough rows for it]
AttnPlan attn_plan(int sms, int D, int group, int max_q, int tokens) {
  AttnPlan a;
  a.grid = sms;
  a.nb = (long long)group * max_q > 8 ? 2 : 1;
  a.counters_off = 256;
  a.partials_off = round_up(a.counters_off + 2 * sizeof(int) * (size_t)sms, 256);
  const size_t part = kv_attn_part_floats(D) * sizeof(float);
  a.firsts_off = a.partials_off + 2 * sms * part;
  a.prompt_off = round_up(a.firsts_off + kKvAttnWarps * sms * part, 256);
  a.bytes = a.prompt_off;
  if ((long long)group * tokens > kPrefillRows) a.bytes += 2 * sms * kv_prefill_part_floats(D) * sizeof(float);
  return a;
}

// Attention of both kinds; words > 0: the new tokens are trees.
marlin_status_t attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int heads, const void* cache,
                          int n_pages, int kv_heads, int head_dim, int page_size, const int32_t* page_table, int max_pages,
                          const int32_t* lengths, const int32_t* q_start, int requests, int tokens, int max_q,
                          const int32_t* tree, int words, float scale, int window, uint16_t* out, void* workspace,
                          size_t workspace_bytes, marlin_stream_t stream) {
  KvAttnParams p{};
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || window < 0 || max_q < 0 || !std::isfinite(scale))
    return MARLIN_ERR_INVALID_ARG;
  marlin_status_t s = make_kv(&p.kv, cache, n_pages, kv_heads, head_dim, page_size, page_table, max_pages, lengths,
                              q_start, requests, tokens, workspace);
  if (s != MARLIN_OK || requests == 0 || tokens == 0) return s;
  if (!q || !out || (words > 0 && !tree)) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(tree, 4)) return MARLIN_ERR_MISALIGNED;
  if (!aligned(q, 16) || !aligned(out, 16) || !strides_ok(q_token_stride, q_head_stride, 8))
    return MARLIN_ERR_MISALIGNED;
  int sms;
  if ((s = current_sms(&sms)) != MARLIN_OK) return s;
  const int group = heads / kv_heads;
  if ((long long)tokens * group > 0x7FFFFFFF) return MARLIN_ERR_UNSUPPORTED;
  const AttnPlan a = attn_plan(sms, head_dim, group, max_q, tokens);
  if (workspace_bytes < a.bytes) return MARLIN_ERR_WORKSPACE_TOO_SMALL;
  {
    static std::mutex lock;
    static bool set[64] = {};
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) return MARLIN_ERR_CUDA;
    std::lock_guard<std::mutex> hold(lock);
    if (dev < 0 || dev >= 64) return MARLIN_ERR_INVALID_ARG;
    if (!set[dev]) {
      if (kv_attn_set_smem_limit() != cudaSuccess || kv_prefill_set_smem_limit() != cudaSuccess) return MARLIN_ERR_CUDA;
      set[dev] = true;
    }
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = q;
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.out = out;
  p.heads = heads;
  p.group = group;
  p.group_magic = group == 1 ? 0ull : ~0ull / (unsigned)group + 1;
  // positions are below 2^30: a window beyond that hides nothing, and position - window stays in 32 bits
  // for the negative positions of a request with more new tokens than its length, too
  p.window = std::min(window, 1 << 30);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.whole_blocks = p.kv.page16 % 4 == 0;
  p.min_rows = 0;
  p.max_rows = 0x7FFFFFFF;
  p.counters = reinterpret_cast<int*>(ws + a.counters_off);
  p.partials = reinterpret_cast<float*>(ws + a.partials_off);
  p.firsts = reinterpret_cast<float*>(ws + a.firsts_off);
  p.timeout_ns = kTimeoutNs;
  p.tree = tree;
  p.tree_words = words;
  // Which kernel: by the query rows that share a key head.  The streaming kernel
  // takes 8 or 16 rows a pass over the cache, the tcgen05 kernel 128.  Where every
  // request has the same number of new tokens one launch serves them all (each
  // kernel is right for any number); else both are launched and each takes its
  // side of the bound, request by request.
  const bool uniform = requests == 1 || (long long)requests * max_q == tokens;
  // (the workspace holds the tcgen05 kernel's parts where all tokens together have enough rows)
  const bool some_large = (long long)(requests == 1 ? tokens : std::min(max_q, tokens)) * group > kPrefillRows;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (some_large) {
    if (!uniform) p.min_rows = kPrefillRows;
    KvAttnParams f = p;
    f.counters = p.counters + a.grid;
    f.partials = reinterpret_cast<float*>(ws + a.prompt_off);
    f.stripes = a.grid;
    const long long items = kv_prefill_items(tokens, requests, kv_heads, group);
    if (items > 0x7FFFFFFF) return MARLIN_ERR_UNSUPPORTED;
    if (launch_kv_prefill(f, head_dim, std::max((int)items, a.grid), st) != cudaSuccess) return MARLIN_ERR_CUDA;
    if (uniform) return MARLIN_OK;
    p.max_rows = kPrefillRows;
  }
  return launch_kv_attn(p, head_dim, a.nb, a.grid, st) == cudaSuccess ? MARLIN_OK : MARLIN_ERR_CUDA;
}

// ---- caches of several layers ---------------------------------------------------------

// Launches `go` for up to kMoveCaches caches at a time.
template <typename Go>
marlin_status_t for_caches(void* const* caches, int count, Go go) {
  for (int c0 = 0; c0 < count; c0 += kMoveCaches) {
    KvCaches c{};
    const int n = std::min(kMoveCaches, count - c0);
    for (int i = 0; i < n; ++i) c.at[i] = static_cast<uint8_t*>(caches[c0 + i]);
    if (go(c, n, c0) != cudaSuccess) return MARLIN_ERR_CUDA;
  }
  return MARLIN_OK;
}

// The layers' caches are all there and do not overlap.
marlin_status_t check_caches(void* const* caches, int count, int n_pages, int hkv, int D, int page) {
  size_t bytes;
  if (count <= 0 || !caches) return MARLIN_ERR_INVALID_ARG;
  if (const marlin_status_t c = marlin_kv_cache_bytes(n_pages, hkv, D, page, &bytes)) return c;
  for (int i = 0; i < count; ++i) {
    if (!caches[i]) return MARLIN_ERR_INVALID_ARG;
    if (!aligned(caches[i], 16)) return MARLIN_ERR_MISALIGNED;
  }
  const auto at = [&](int i) { return reinterpret_cast<uintptr_t>(caches[i]); };
  uintptr_t top = at(0);  // the highest so far
  for (int i = 1; i < count; ++i) {
    if (at(i) >= top && at(i) - top >= bytes) {  // as they come from an allocator, mostly
      top = at(i);
      continue;
    }
    top = std::max(top, at(i));
    for (int j = 0; j < i; ++j)
      if ((at(i) > at(j) ? at(i) - at(j) : at(j) - at(i)) < bytes) return MARLIN_ERR_INVALID_ARG;
  }
  return MARLIN_OK;
}

}  // namespace

extern "C" {

marlin_status_t marlin_lora_workspace_bytes(int M, int K, int N, int group, int r, int device, size_t* bytes) {
  if (!bytes || M < 0 || r <= 0) return MARLIN_ERR_INVALID_ARG;
  if (r % 8 != 0 || r > kLoraMaxRank) return MARLIN_ERR_UNSUPPORTED;
  LoraSizes z;
  const marlin_status_t s = lora_sizes(M, K, N, group, r, device, &z);
  if (s == MARLIN_OK) *bytes = z.total;
  return s;
}

marlin_status_t marlin_lora_gemm(const uint16_t* X, const void* packed, const uint16_t* scales, const int32_t* zeros,
                                 const uint16_t* A, const uint16_t* B, const float* scaling, const int32_t* index,
                                 int adapters, int r, uint16_t* Y, int M, int K, int N, int group, void* workspace,
                                 size_t workspace_bytes, marlin_stream_t stream) {
  if (M < 0 || r <= 0 || adapters <= 0) return MARLIN_ERR_INVALID_ARG;
  if (const marlin_status_t c = marlin_packed_layout(K, N, group, 0, nullptr, nullptr, nullptr)) return c;
  if (r % 8 != 0 || r > kLoraMaxRank) return MARLIN_ERR_UNSUPPORTED;
  if (M == 0) return MARLIN_OK;
  if (!X || !packed || !scales || !A || !B || !scaling || !index || !Y || !workspace) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(packed, 16) || !aligned(scales, 16) || !aligned(zeros, 16) || !aligned(A, 16) ||
      !aligned(B, 16) || !aligned(scaling, 4) || !aligned(index, 4) || !aligned(Y, 16) || !aligned(workspace, 16))
    return MARLIN_ERR_MISALIGNED;
  int dev, sms;
  if (cudaGetDevice(&dev) != cudaSuccess) return MARLIN_ERR_CUDA;
  marlin_status_t s = static_cast<marlin_status_t>(device_sms(dev, &sms));
  if (s != MARLIN_OK) return s;
  LoraSizes z;
  if ((s = lora_sizes(M, K, N, group, r, dev, &z)) != MARLIN_OK) return s;
  if (workspace_bytes < z.total) return MARLIN_ERR_WORKSPACE_TOO_SMALL;
  LoraParams p{};
  p.x = X;
  p.a = A;
  p.b = B;
  p.scaling = scaling;
  p.index = index;
  p.y = Y;
  p.v = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + z.v_off);
  p.unit = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + z.unit_off);
  p.arrived = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + z.arrived_off);
  p.rp = (int)round_up(r, 16);
  p.status = static_cast<int*>(workspace);
  p.M = M;
  p.K = K;
  p.N = N;
  p.r = r;
  p.adapters = adapters;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (lora_two_kernels(M, r) && launch_lora(p, 0, sms, st) != cudaSuccess) return MARLIN_ERR_CUDA;
  s = marlin_gemm(X, packed, scales, zeros, Y, M, K, N, group, workspace, z.gemm, stream);
  if (s != MARLIN_OK) return s;
  return launch_lora(p, 1, sms, st) == cudaSuccess ? MARLIN_OK : MARLIN_ERR_CUDA;
}

marlin_status_t marlin_kv_cache_bytes(int n_pages, int kv_heads, int head_dim, int page_size, size_t* bytes) {
  if (!bytes) return MARLIN_ERR_INVALID_ARG;
  if (const marlin_status_t c = check_cache(n_pages, kv_heads, head_dim, page_size)) return c;
  *bytes = (size_t)n_pages * kv_heads * (page_size / kGranule) * kv_granule_bytes(head_dim);
  return MARLIN_OK;
}

marlin_status_t marlin_kv_workspace_bytes(int heads, int kv_heads, int head_dim, int requests, int tokens, int device,
                                          size_t* bytes) {
  if (!bytes || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || requests < 0 || tokens < 0)
    return MARLIN_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MARLIN_ERR_UNSUPPORTED;
  int sms;
  const marlin_status_t s = static_cast<marlin_status_t>(device_sms(device, &sms));
  if (s != MARLIN_OK) return s;
  *bytes = attn_plan(sms, head_dim, heads / kv_heads, 1, tokens).bytes;
  return MARLIN_OK;
}

marlin_status_t marlin_kv_append(const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                                 int64_t v_token_stride, int64_t v_head_stride, void* cache, int n_pages, int kv_heads,
                                 int head_dim, int page_size, const int32_t* page_table, int max_pages,
                                 const int32_t* lengths, const int32_t* q_start, int requests, int tokens,
                                 void* workspace, marlin_stream_t stream) {
  return kv_copy(true, const_cast<uint16_t*>(k), k_token_stride, k_head_stride, const_cast<uint16_t*>(v),
                 v_token_stride, v_head_stride, cache, n_pages, kv_heads, head_dim, page_size, page_table, max_pages,
                 lengths, q_start, requests, tokens, workspace, stream);
}

marlin_status_t marlin_kv_read(uint16_t* k, uint16_t* v, const void* cache, int n_pages, int kv_heads, int head_dim,
                               int page_size, const int32_t* page_table, int max_pages, const int32_t* lengths,
                               const int32_t* q_start, int requests, int tokens, void* workspace,
                               marlin_stream_t stream) {
  const int64_t ts = (int64_t)kv_heads * head_dim;
  return kv_copy(false, k, ts, head_dim, v, ts, head_dim, cache, n_pages, kv_heads, head_dim, page_size, page_table,
                 max_pages, lengths, q_start, requests, tokens, workspace, stream);
}

marlin_status_t marlin_kv_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int heads,
                                    const void* cache, int n_pages, int kv_heads, int head_dim, int page_size,
                                    const int32_t* page_table, int max_pages, const int32_t* lengths,
                                    const int32_t* q_start, int requests, int tokens, int max_q, float scale,
                                    int window, uint16_t* out, void* workspace, size_t workspace_bytes,
                                    marlin_stream_t stream) {
  return attention(q, q_token_stride, q_head_stride, heads, cache, n_pages, kv_heads, head_dim, page_size, page_table,
                   max_pages, lengths, q_start, requests, tokens, max_q, nullptr, 0, scale, window, out, workspace,
                   workspace_bytes, stream);
}

marlin_status_t marlin_kv_tree_attention(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int heads,
                                         const void* cache, int n_pages, int kv_heads, int head_dim, int page_size,
                                         const int32_t* page_table, int max_pages, const int32_t* lengths,
                                         const int32_t* q_start, int requests, int tokens, int max_q,
                                         const int32_t* mask, int words, float scale, int window, uint16_t* out,
                                         void* workspace, size_t workspace_bytes, marlin_stream_t stream) {
  if (words <= 0) return MARLIN_ERR_INVALID_ARG;
  return attention(q, q_token_stride, q_head_stride, heads, cache, n_pages, kv_heads, head_dim, page_size, page_table,
                   max_pages, lengths, q_start, requests, tokens, max_q, mask, words, scale, window, out, workspace,
                   workspace_bytes, stream);
}

marlin_status_t marlin_kv_tree(const int32_t* parents, const int32_t* lengths, const int32_t* q_start, int requests,
                               int tokens, int words, int32_t* mask, int32_t* positions, void* workspace,
                               marlin_stream_t stream) {
  if (requests < 0 || tokens < 0 || words <= 0) return MARLIN_ERR_INVALID_ARG;
  if (requests == 0 || tokens == 0) return MARLIN_OK;
  if (!parents || !lengths || !q_start || !mask || !positions || !workspace) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(parents, 4) || !aligned(lengths, 4) || !aligned(q_start, 4) || !aligned(mask, 4) || !aligned(positions, 4) ||
      !aligned(workspace, 16))
    return MARLIN_ERR_MISALIGNED;
  KvParams p{};
  p.B = requests;
  p.T = tokens;
  p.lens = lengths;
  p.q_start = q_start;
  p.status = static_cast<int*>(workspace);
  p.max_pages = 1;  // lengths up to 2^30, as in any cache
  p.page = 1 << 30;
  return launch_kv_tree(p, parents, words, mask, positions, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MARLIN_OK
             : MARLIN_ERR_CUDA;
}

marlin_status_t marlin_kv_rope_append(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride, int heads,
                                      const uint16_t* k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t* v,
                                      int64_t v_token_stride, int64_t v_head_stride, const int32_t* positions, int axes,
                                      const float* table, int table_rows, int rot, int interleaved,
                                      const uint8_t* axis_of_pair, uint16_t* q_out, int64_t out_token_stride,
                                      int64_t out_head_stride, void* cache, int n_pages, int kv_heads, int head_dim,
                                      int page_size, const int32_t* page_table, int max_pages, const int32_t* lengths,
                                      const int32_t* q_start, int requests, int tokens, void* workspace,
                                      marlin_stream_t stream) {
  KvRopeParams p{};
  if (heads <= 0 || axes <= 0 || table_rows <= 0 || rot <= 0 || rot > head_dim) return MARLIN_ERR_INVALID_ARG;
  const marlin_status_t s = make_kv(&p.kv, cache, n_pages, kv_heads, head_dim, page_size, page_table, max_pages, lengths,
                                    q_start, requests, tokens, workspace);
  if (s != MARLIN_OK) return s;
  if (axes > kRopeAxes || rot % (head_dim / 8) != 0) return MARLIN_ERR_UNSUPPORTED;
  if (axes > 1 && !axis_of_pair) return MARLIN_ERR_INVALID_ARG;
  p.grouped = 1;
  for (int j = 0; axis_of_pair && j < rot / 2; ++j) {
    if (axis_of_pair[j] >= axes) return MARLIN_ERR_INVALID_ARG;
    p.axis[j / 32] |= (unsigned long long)axis_of_pair[j] << (2 * (j % 32));
    if (j % (head_dim / 32) != 0 && axis_of_pair[j] != axis_of_pair[j - 1]) p.grouped = 0;
  }
  if (requests == 0 || tokens == 0) return MARLIN_OK;
  if (!q || !k || !v || !positions || !table || !q_out) return MARLIN_ERR_INVALID_ARG;
  if (out_token_stride >= 0 && out_head_stride >= 0 &&
      !rows_apart(out_token_stride, out_head_stride, tokens, heads, head_dim))
    return MARLIN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(positions, 4) ||
      !aligned(table, 16) || !strides_ok(q_token_stride, q_head_stride, 8) || !strides_ok(k_token_stride, k_head_stride, 8) ||
      !strides_ok(v_token_stride, v_head_stride, 8) || !strides_ok(out_token_stride, out_head_stride, 8))
    return MARLIN_ERR_MISALIGNED;
  p.q = q;
  p.q_ts = q_token_stride;
  p.q_hs = q_head_stride;
  p.heads = heads;
  p.k = k;
  p.k_ts = k_token_stride;
  p.k_hs = k_head_stride;
  p.v = v;
  p.v_ts = v_token_stride;
  p.v_hs = v_head_stride;
  p.q_out = q_out;
  p.o_ts = out_token_stride;
  p.o_hs = out_head_stride;
  p.positions = positions;
  p.axes = axes;
  p.table = table;
  p.table_rows = table_rows;
  p.rot = rot;
  int sms;
  if (const marlin_status_t c = current_sms(&sms)) return c;
  return launch_kv_rope_append(p, head_dim, interleaved != 0, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MARLIN_OK
             : MARLIN_ERR_CUDA;
}

marlin_status_t marlin_kv_compact(void* const* caches, int count, int n_pages, int kv_heads, int head_dim, int page_size,
                                  const int32_t* page_table, int max_pages, const int32_t* into, int into_pages,
                                  const int32_t* lengths, const int32_t* q_start, const int32_t* index,
                                  const int32_t* kept, int32_t* new_lengths, int requests, int tokens, int max_q,
                                  void* workspace, marlin_stream_t stream) {
  KvCompactParams p{};
  if (max_q < 0 || (into && into_pages <= 0)) return MARLIN_ERR_INVALID_ARG;
  if (const marlin_status_t c = check_caches(caches, count, n_pages, kv_heads, head_dim, page_size)) return c;
  const marlin_status_t s = make_kv(&p.kv, caches[0], n_pages, kv_heads, head_dim, page_size, page_table, max_pages, lengths,
                                    q_start, requests, tokens, workspace);
  if (s != MARLIN_OK) return s;
  if (into && (long long)into_pages * page_size > (1ll << 30)) return MARLIN_ERR_UNSUPPORTED;
  if (requests == 0) return MARLIN_OK;
  if (!lengths || !q_start || !page_table || !workspace || (!index && tokens > 0) || !kept || !new_lengths)
    return MARLIN_ERR_INVALID_ARG;
  if (!aligned(into, 4) || !aligned(index, 4) || !aligned(kept, 4) || !aligned(new_lengths, 4) || !aligned(lengths, 4))
    return MARLIN_ERR_MISALIGNED;
  if (tokens == 0)
    return cudaMemcpyAsync(new_lengths, lengths, (size_t)requests * sizeof(int32_t), cudaMemcpyDeviceToDevice,
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MARLIN_OK
               : MARLIN_ERR_CUDA;
  p.into = into;
  p.into_pages = into_pages;
  p.index = index;
  p.kept = kept;
  p.max_q = std::min(max_q, tokens);
  int sms;
  if (const marlin_status_t c = current_sms(&sms)) return c;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return for_caches(caches, count, [&](const KvCaches& c, int n, int c0) {
    p.caches = n;
    p.new_lens = c0 == 0 ? new_lengths : nullptr;
    return launch_kv_compact(p, c, head_dim, sms, st);
  });
}

marlin_status_t marlin_kv_copy_pages(void* const* caches, int count, int n_pages, int kv_heads, int head_dim,
                                     int page_size, const int32_t* src, const int32_t* dst, int pairs, void* workspace,
                                     marlin_stream_t stream) {
  if (pairs < 0) return MARLIN_ERR_INVALID_ARG;
  if (const marlin_status_t c = check_caches(caches, count, n_pages, kv_heads, head_dim, page_size)) return c;
  size_t bytes;
  if (const marlin_status_t c = marlin_kv_cache_bytes(1, kv_heads, head_dim, page_size, &bytes)) return c;
  if (pairs == 0) return MARLIN_OK;
  if (!src || !dst || !workspace) return MARLIN_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(workspace, 16)) return MARLIN_ERR_MISALIGNED;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return for_caches(caches, count, [&](const KvCaches& c, int n, int) {
    return launch_kv_copy_pages(c, n, n_pages, (long long)bytes, src, dst, pairs, static_cast<int*>(workspace), st);
  });
}

}  // extern "C"
