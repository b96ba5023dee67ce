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
  KvAttnParams p{};
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 || window < 0 || max_q < 0 || !std::isfinite(scale))
    return MARLIN_ERR_INVALID_ARG;
  marlin_status_t s = make_kv(&p.kv, cache, n_pages, kv_heads, head_dim, page_size, page_table, max_pages, lengths,
                              q_start, requests, tokens, workspace);
  if (s != MARLIN_OK || requests == 0 || tokens == 0) return s;
  if (!q || !out) return MARLIN_ERR_INVALID_ARG;
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
  // Which kernel: by the query rows that share a key head.  The streaming kernel
  // takes 8 or 16 rows a pass over the cache, the tcgen05 kernel 128.  Where every
  // request has the same number of new tokens one launch serves them all (each
  // kernel is right for any number); else both are launched and each takes its
  // side of the bound, request by request.
  const bool uniform = requests == 1 || (long long)requests * max_q == tokens;
  const bool some_large = (long long)(requests == 1 ? tokens : max_q) * group > kPrefillRows;
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

}  // extern "C"
