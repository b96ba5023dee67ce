// kv_move.cu -- moving what the caches of a model's layers hold: the kept ones of a request's new tokens
// together (after a tree of drafted tokens was verified, or to drop tokens of a long context), and whole
// pages.  One launch serves the caches of all layers, which share pages, lengths and indexes.
#include <algorithm>

#include "kv.cuh"

namespace w4a16 {

namespace {

// ---- kept tokens ---------------------------------------------------------------------------------
// Position first + i of request b takes what position first + index[i] held, for i < kept[b], first the
// position of the first new token.
//
// Bound: the stream, kept entries of 2 (D/2 + 4) bytes out of and into every head of every cache, and the
// latency of a chain of three loads (index, page, entry).  A warp builds a granule of 16 positions in
// registers, all of its loads in flight, and writes it in whole lines: keys are moved in 16-byte pieces;
// a word of values pairs two tokens, so that a lane loads the words of both its tokens and takes a half of
// each (kv.cuh).  Where the kept tokens stay in their pages, W warps (a unit) take a request's head in
// rounds of W granules, loads before stores: index[i] ascends, so no round reads what one before has
// written, and a barrier between a round's loads and stores keeps it from overwriting what is still read.
// Where tokens come from is the same for every head of every cache.  Where they go to other pages and there is
// work for every warp, a warp finds it once for up to 8 heads, two of them in flight: 38,668 of 76,825 tokens, 8 heads
// of 128 channels, 20.6 us (84 MB out and in, 4.1 TB/s; 25 where nothing of it is in L2), of which the look at the indexes
// is 2.5.  Without that look: 20.5 with one in flight, 26.3 a head a warp, 23 with four in flight (their registers leave
// fewer warps).  Of few tokens a head a warp is faster: half of 500 of 2 requests, with the read back, 6.7 against 9.2 us, and
// in place, where warps that moved several were up to 15% slower.  A kept token's values share their 32-byte
// sectors with up to 15 others, so that more is read than kept: 5 tokens of each of 40 requests in place, in 32 caches,
// 10.6 us (7 MB kept, 34 read).  In place few heads are few CTAs, and their rounds a chain: the 38,668 tokens 333 us.
constexpr int kMoveThreads = 256, kMoveWarps = kMoveThreads / 32;

// What warps read of a request, checked.
struct Kept {
  KvSeq s;
  int first, kept;
};
__device__ __forceinline__ Kept kept_of(const KvCompactParams& p, int b, bool report) {
  Kept k;
  k.s = kv_seq(p.kv, b, report);
  k.first = k.s.len - k.s.nq;
  k.kept = p.kept[b];
  if (k.first < 0) {
    if (report) kv_fail(p.kv, kKvSiteLen);
    k.kept = -1;
  } else if (k.kept < 0 || k.kept > k.s.nq) {
    if (report) kv_fail(p.kv, kKvSiteIndex);
    k.kept = -1;
  }
  return k;  // kept < 0: nothing is moved
}

// By a warp: whether index ascends strictly, within the new tokens.
__device__ __forceinline__ bool ascends(const KvCompactParams& p, const Kept& k) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  for (int i = lane; i < k.kept; i += 32) {
    const int at = p.index[k.s.q0 + i], before = i ? p.index[k.s.q0 + i - 1] : -1;
    ok = ok && at > before && at < k.s.nq;
  }
  return __all_sync(0xffffffffu, ok);
}

// Byte offset of a position's granule in a cache, of key head 0; -1 for a page that does not exist.
template <int D>
__device__ __forceinline__ long long granule_at(const KvParams& p, const int* row, int pages, int pos) {
  const int g16 = pos >> 4, pi = kv_div_page(p, g16);
  const int page = pi < pages ? row[pi] : -1;
  if (page < 0 || page >= p.n_pages) {
    kv_fail(p, kKvSitePage);
    return -1;
  }
  return page * p.page_bytes + (long long)(g16 - pi * p.page16) * kv_granule_bytes(D);
}

// Where the 16 tokens of a granule come from: lane s < 16 has token s; lanes of tokens that are not
// written have from < 0.
struct Plan {
  long long from, to;  // offsets of this lane's source granule, of the granule itself
  int tok;             // the source's place in its granule
};

template <int D>
__device__ __forceinline__ Plan plan_granule(const KvCompactParams& p, const Kept& k, int b, int granule) {
  const int lane = threadIdx.x & 31, pos = granule * 16 + lane, i = pos - k.first;
  Plan m{-1, -1, 0};
  const bool mine = lane < 16 && i >= 0 && i < k.kept;
  if (mine) {
    const int at = p.index[k.s.q0 + i];
    if (at < 0 || at >= k.s.nq) {  // (not unless it has changed since all indexes were looked at)
      kv_fail(p.kv, kKvSiteIndex);
    } else {
      m.from = granule_at<D>(p.kv, p.kv.table + (long long)b * p.kv.max_pages, p.kv.max_pages, k.first + at);
      m.tok = (k.first + at) & 15;
    }
  }
  const int lead = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  if (lead >= 0) {
    if (lane == lead)
      m.to = p.into ? granule_at<D>(p.kv, p.into + (long long)b * p.into_pages, p.into_pages, pos)
                    : granule_at<D>(p.kv, p.kv.table + (long long)b * p.kv.max_pages, p.kv.max_pages, pos);
    m.to = __shfl_sync(0xffffffffu, m.to, lead);
  }
  return m;
}

template <int N>
__device__ __forceinline__ void get_words(const uint8_t* at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  }
}

// A granule's bytes in a warp's registers.
template <int D>
struct Granule {
  static constexpr int NK = D / 64, CW = D / 32;  // 16-byte pieces of keys, words of a lane's values in a half
  uint4 k[NK];
  uint32_t v[2][CW];
  uint2 s;
  uint32_t live;  // tokens that are written
};

// Where a lane's pieces of a granule come from, offsets from the beginning of a head.
template <int D>
struct Source {
  static constexpr int PK = D / 32;  // 16-byte pieces of a token's keys
  long long k[D / 64], v[2][2], s;
  uint32_t pick[2];  // which halves of the two tokens' words
  uint32_t live;     // tokens that are written
};

template <int D>
__device__ __forceinline__ Source<D> source_of(const Plan& m) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  Source<D> o;
  o.live = __ballot_sync(0xffffffffu, m.from >= 0 && m.to >= 0);
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const int piece = j * 32 + lane, s = piece / o.PK;
    const long long from = __shfl_sync(0xffffffffu, m.from, s);
    const int tok = __shfl_sync(0xffffffffu, m.tok, s);
    o.k[j] = from + tok * (D / 2) + (piece % o.PK) * 16;
  }
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    int odd[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int s = 8 * hf + 2 * c + e;
      const long long from = __shfl_sync(0xffffffffu, m.from, s);
      const int tok = __shfl_sync(0xffffffffu, m.tok, s);
      odd[e] = tok & 1;
      o.v[hf][e] = from + 8 * D + (tok >> 3) * (4 * D) + (4 * g + ((tok & 7) >> 1)) * (D / 8);
    }
    o.pick[hf] = (odd[0] ? 0x32u : 0x10u) | (odd[1] ? 0x7600u : 0x5400u);
  }
  o.s = m.from + 16 * D + 8 * m.tok;
  return o;
}

template <int D>
__device__ __forceinline__ void load_granule(const uint8_t* head, const Source<D>& o, Granule<D>& r) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  r.live = o.live;
#pragma unroll
  for (int j = 0; j < Granule<D>::NK; ++j)
    if ((o.live >> ((j * 32 + lane) / o.PK)) & 1u) r.k[j] = *reinterpret_cast<const uint4*>(head + o.k[j]);
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    uint32_t w[2][Granule<D>::CW];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int i = 0; i < Granule<D>::CW; ++i) w[e][i] = 0u;
      if ((o.live >> (8 * hf + 2 * c + e)) & 1u) get_words<Granule<D>::CW>(head + o.v[hf][e], w[e]);
    }
#pragma unroll
    for (int i = 0; i < Granule<D>::CW; ++i) r.v[hf][i] = __byte_perm(w[0][i], w[1][i], o.pick[hf]);
  }
  if (lane < 16 && ((o.live >> lane) & 1u)) r.s = *reinterpret_cast<const uint2*>(head + o.s);
}

template <int D>
__device__ __forceinline__ void store_granule(uint8_t* head, long long at, const Granule<D>& r) {
  constexpr int PK = D / 32, CW = Granule<D>::CW;
  const int lane = threadIdx.x & 31, c = lane & 3;
  if (r.live == 0) return;
  uint8_t* to = head + at;
#pragma unroll
  for (int j = 0; j < Granule<D>::NK; ++j) {
    const int piece = j * 32 + lane;
    if ((r.live >> (piece / PK)) & 1u) *reinterpret_cast<uint4*>(to + piece * 16) = r.k[j];
  }
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    const uint32_t both = (r.live >> (8 * hf + 2 * c)) & 3u;
    uint8_t* row = to + 8 * D + hf * (4 * D) + lane * (D / 8);
    if (both == 3u) {
      if constexpr (CW == 4) *reinterpret_cast<uint4*>(row) = make_uint4(r.v[hf][0], r.v[hf][1], r.v[hf][2], r.v[hf][3]);
      else *reinterpret_cast<uint2*>(row) = make_uint2(r.v[hf][0], r.v[hf][1]);
    } else if (both) {  // the other token of the words is not to be touched
      const int e = both >> 1;
#pragma unroll
      for (int i = 0; i < CW; ++i) *reinterpret_cast<uint16_t*>(row + 4 * i + 2 * e) = (uint16_t)(r.v[hf][i] >> (16 * e));
    }
  }
  if (lane < 16 && ((r.live >> lane) & 1u)) *reinterpret_cast<uint2*>(to + 16 * D + 8 * lane) = r.s;
}

// The kept tokens stay in their pages.  W warps a unit: (request, cache, head), heads fastest.
template <int D, int W>
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const KvCompactParams p, const __grid_constant__ KvCaches caches) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long unit = (long long)blockIdx.x * (kMoveWarps / W) + warp / W;
  const int heads = p.caches * p.kv.hkv;
  if (unit >= (long long)heads * p.kv.B) return;  // a whole unit
  const int b = (int)(unit / heads), at = (int)(unit - (long long)b * heads), cache = at / p.kv.hkv;
  const bool speaks = at == 0 && warp % W == 0;  // one warp of the request
  Kept k = kept_of(p, b, speaks && lane == 0);
  if (k.kept > 0 && !ascends(p, k)) {
    if (speaks && lane == 0) kv_fail(p.kv, kKvSiteIndex);
    k.kept = -1;
  }
  if (speaks && lane == 0 && p.new_lens) p.new_lens[b] = k.kept < 0 ? p.kv.lens[b] : k.first + k.kept;
  if (k.kept <= 0) return;
  uint8_t* head = caches.at[cache] + (at - cache * p.kv.hkv) * p.kv.head_bytes;
  const int g_end = (k.first + k.kept + 15) >> 4;
  for (int g0 = k.first >> 4; g0 < g_end; g0 += W) {
    const int granule = g0 + warp % W;
    Granule<D> r;
    r.live = 0;
    Plan m{-1, -1, 0};
    if (granule < g_end) {
      m = plan_granule<D>(p, k, b, granule);
      load_granule<D>(head, source_of<D>(m), r);
    }
    if constexpr (W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(W * 32) : "memory");
    store_granule<D>(head, m.to, r);
  }
}

// The kept tokens go to other pages: a warp has granules of `run` of all caches' heads, H in flight.  Nothing of a
// request with an index outside its new tokens is moved, so that all of its indexes are looked at before a warp's first
// store, under its first loads: by every warp (p.look) where they are few, else by a kernel before (kv_index_kernel),
// which reports what is outside; while nothing is reported there is nothing to find, and until what was reported is
// read every warp looks.
constexpr int kMostHeads = 8;
// New tokens of a request.  Half of the tokens of 2 requests of 250 3.5 us where every warp looks, 4.5 with a kernel
// before; of 1000 4.5 / 5.0, of 2000 5.8 / 5.2, of 4000 9.0 / 6.4, of 38,000 58.7 / 21.7 (20.0 if nobody looked); 8 heads
// of 128 channels.
constexpr int kLookMost = 1024;

constexpr int kIndexes = 8;  // of a thread, in flight
__device__ __forceinline__ bool inside(const KvCompactParams& p, const Kept& k, long long i0, int step) {
  bool ok = true;
#pragma unroll
  for (int j = 0; j < kIndexes; ++j) {
    const long long i = i0 + j * step;
    const int at = i < k.kept ? p.index[k.s.q0 + i] : 0;
    ok &= (uint32_t)at < (uint32_t)k.s.nq;
  }
  return ok;
}

__global__ void __launch_bounds__(kMoveThreads) kv_index_kernel(const KvCompactParams p, int ctas) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int b = blockIdx.x / ctas;
  const Kept k = kept_of(p, b, false);  // (counts and lengths that do not fit are the next kernel's to report)
  constexpr long long kChunk = kMoveThreads * kIndexes;
  bool ok = true;
  for (long long i = blockIdx.x % ctas * kChunk + threadIdx.x; i < k.kept; i += ctas * kChunk)
    ok &= inside(p, k, i, kMoveThreads);
  if (!ok) kv_fail(p.kv, kKvSiteIndex);
}

template <int D, int H>
__global__ void __launch_bounds__(kMoveThreads) kv_gather_kernel(const KvCompactParams p, const __grid_constant__ KvCaches caches,
                                                                 int ctas, int run) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int x = blockIdx.x % ctas, unit = blockIdx.x / ctas;  // of a run's CTAs
  const int heads = p.caches * p.kv.hkv, runs = (heads + run - 1) / run, b = unit / runs, at = (unit - b * runs) * run;
  const bool speaks = at == 0 && x == 0 && threadIdx.x == 0;
  const int reported = p.look ? 1 : __ldcg(p.kv.status);
  const Kept k = kept_of(p, b, speaks);
  if (k.kept <= 0) {
    if (speaks && p.new_lens) p.new_lens[b] = k.kept < 0 ? p.kv.lens[b] : k.first;
    return;
  }
  const int g_end = (k.first + k.kept + 15) >> 4, first_cache = at / p.kv.hkv, first_head = at - first_cache * p.kv.hkv;
  bool sure = false;  // that all indexes are inside
  for (int granule = (k.first >> 4) + x * kMoveWarps + (threadIdx.x >> 5); granule < g_end; granule += ctas * kMoveWarps) {
    const Plan m = plan_granule<D>(p, k, b, granule);
    const Source<D> o = source_of<D>(m);
    int cache = first_cache, h = first_head;
    for (int left = min(run, heads - at); left > 0; left -= H) {
      uint8_t* head[H];
      Granule<D> r[H];
#pragma unroll
      for (int i = 0; i < H; ++i)
        if (i < left) {
          head[i] = caches.at[cache] + h * p.kv.head_bytes;
          load_granule<D>(head[i], o, r[i]);
          if (++h == p.kv.hkv) {
            h = 0;
            ++cache;
          }
        }
      if (!sure) {
        bool ok = true;
        if (__any_sync(0xffffffffu, reported != 0))
          for (long long i = threadIdx.x & 31; i < k.kept; i += 32 * kIndexes) ok &= inside(p, k, i, 32);
        sure = __all_sync(0xffffffffu, ok);
        if (speaks && !sure) kv_fail(p.kv, kKvSiteIndex);
        if (speaks && p.new_lens) p.new_lens[b] = sure ? k.first + k.kept : p.kv.lens[b];  // (its warp has the first granule)
        if (!sure) return;
      }
#pragma unroll
      for (int i = 0; i < H; ++i)
        if (i < left) store_granule<D>(head[i], m.to, r[i]);
    }
  }
}

// ---- pages -------------------------------------------------------------------------------------------
// Bound: the stream, a page's bytes in and out for every pair and cache.  A CTA copies 16 KB, four loads
// of 16 bytes in flight a thread.  Measured: 45 pages of 70 KB in 32 caches 31.3 us, 6.4 TB/s (94% of the card's
// copy rate); one page in 32 caches 2.2 us.
constexpr int kPageThreads = 256, kPageVecs = 4, kPageChunk = kPageThreads * kPageVecs * 16;

__global__ void __launch_bounds__(kPageThreads) kv_copy_pages_kernel(const __grid_constant__ KvCaches caches, int n_caches,
                                                                     int n_pages, long long page_bytes, int chunks,
                                                                     const int* src, const int* dst, int* status) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  const int chunk = blockIdx.x % chunks, rest = blockIdx.x / chunks, cache = rest % n_caches, pair = rest / n_caches;
  const int from = src[pair], to = dst[pair];
  if (from < 0) return;  // no pair
  if (from >= n_pages || to < 0 || to >= n_pages) {
    if (chunk == 0 && cache == 0 && threadIdx.x == 0) {
      atomicCAS(status + 1, 0, kKvSitePage);
      atomicOr(status, kStatusBounds);
    }
    return;
  }
  const uint4* in = reinterpret_cast<const uint4*>(caches.at[cache] + from * page_bytes);
  uint4* out = reinterpret_cast<uint4*>(caches.at[cache] + to * page_bytes);
  const int vecs = (int)(page_bytes / 16), v0 = chunk * (kPageChunk / 16) + threadIdx.x;
  uint4 v[kPageVecs];
#pragma unroll
  for (int i = 0; i < kPageVecs; ++i)
    if (v0 + i * kPageThreads < vecs) v[i] = in[v0 + i * kPageThreads];
#pragma unroll
  for (int i = 0; i < kPageVecs; ++i)
    if (v0 + i * kPageThreads < vecs) out[v0 + i * kPageThreads] = v[i];
}

template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), long long ctas, int threads, cudaStream_t stream, Args... args) {
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D>
cudaError_t compact(const KvCompactParams& p, const KvCaches& c, int sms, cudaStream_t stream) {
  const long long units = (long long)p.kv.B * p.caches * p.kv.hkv;
  const long long granules = ((long long)p.max_q + 15) / 16 + 1;  // at most, of a request
  if (p.into) {
    const long long ctas = (granules + kMoveWarps - 1) / kMoveWarps;
    const int heads = p.caches * p.kv.hkv;
    KvCompactParams f = p;
    f.look = p.max_q <= kLookMost;
    if (!f.look && p.new_lens) {  // the first of several launches
      const long long looks = (p.max_q + kMoveThreads * kIndexes - 1ll) / (kMoveThreads * kIndexes);
      const cudaError_t e = launch(kv_index_kernel, p.kv.B * looks, kMoveThreads, stream, p, (int)looks);
      if (e != cudaSuccess) return e;
    }
    // 32 warps an SM at least, as many as fit where a head is a warp's
    const int run = (int)std::min<long long>(std::max<long long>(units * granules / (32ll * sms), 1), kMostHeads);
    return launch(run == 1 ? kv_gather_kernel<D, 1> : kv_gather_kernel<D, 2>, p.kv.B * ((heads + run - 1ll) / run) * ctas,
                  kMoveThreads, stream, f, c, (int)ctas, run);
  }
  // a warp a head where few tokens can be kept (more are served by it in more rounds), else a CTA
  if (granules <= 16) return launch(kv_compact_kernel<D, 1>, (units + kMoveWarps - 1) / kMoveWarps, kMoveThreads, stream, p, c);
  return launch(kv_compact_kernel<D, 8>, units, kMoveThreads, stream, p, c);
}

}  // namespace

cudaError_t launch_kv_compact(const KvCompactParams& p, const KvCaches& c, int D, int sms, cudaStream_t stream) {
  return D == 128 ? compact<128>(p, c, sms, stream) : compact<64>(p, c, sms, stream);
}

cudaError_t launch_kv_copy_pages(const KvCaches& c, int caches, int n_pages, long long page_bytes, const int* src,
                                 const int* dst, int pairs, int* status, cudaStream_t stream) {
  const int chunks = (int)((page_bytes + kPageChunk - 1) / kPageChunk);
  const long long ctas = (long long)chunks * caches * pairs;
  return launch(kv_copy_pages_kernel, ctas, kPageThreads, stream, c, caches, n_pages, page_bytes, chunks, src, dst, status);
}

}  // namespace w4a16
