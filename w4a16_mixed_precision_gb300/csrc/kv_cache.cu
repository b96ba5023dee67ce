// kv_cache.cu -- writing new keys and values into the 4-bit paged cache, with or
// without rotating queries and keys by their positions first, and reading cached
// values back as fp16.
//
// Bound: both are streams, 4 D bytes of fp16 in (or out) and D + 8 bytes of
// cache per token and head.  Quantising costs about ten operations a channel,
// so the work per vector is kept low: eight lanes share a vector (three shuffle
// steps for its minimum and maximum, taken on packed fp16), a warp takes four
// consecutive tokens of one head, keys and values, with all loads in flight
// before the look-ups of their places; two tokens that share a word of values
// write it together.  Measured with 128 channels, 8 heads: 10,740 tokens (56 MB) are
// written in 19.3 us, 2.9 TB/s, and read back in 13.9 us, 4.0 TB/s (43 and 60% of the
// card's copy rate); 48 tokens in 4.1 and 3.3 us.  Writing issues an instruction in 68%
// of the cycles; fewer for the codes (sums instead of shifts) changed nothing, so what
// is left is the loads' latency under one short task per warp.
#include <algorithm>

#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr int kKvThreads = 256;
constexpr int kTokens = 4;  // of a warp

// Where row t of the new tokens, of request b, lives at head h: its granule, and its place in it;
// nullptr if the inputs give it none.
template <int D>
__device__ __forceinline__ uint8_t* kv_place_of(const KvParams& p, int t, int b, const KvSeq& s, int h, int* in_granule) {
  if (t < s.q0 || t >= s.q0 + s.nq) return nullptr;
  const int pos = s.len - (s.q0 + s.nq - t);
  if (pos < 0) {
    kv_fail(p, kKvSiteLen);
    return nullptr;
  }
  const int g16 = pos >> 4;
  const int pi = kv_div_page(p, g16);
  const int page = p.table[(long long)b * p.max_pages + pi];
  if (page < 0 || page >= p.n_pages) {
    kv_fail(p, kKvSitePage);
    return nullptr;
  }
  *in_granule = pos & 15;
  return p.cache + page * p.page_bytes + h * p.head_bytes + (long long)(g16 - pi * p.page16) * kv_granule_bytes(D);
}
template <int D>
__device__ __forceinline__ uint8_t* kv_place(const KvParams& p, int t, int h, int* in_granule) {
  const int b = kv_owner(p, t);
  return kv_place_of<D>(p, t, b, kv_seq(p, b, true), h, in_granule);
}

__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ uint32_t pair_bits(__half a, __half b) { return bits(__halves2half2(a, b)); }

// Codes of CPL channels (pairs in x), and the vector's scale and offset; its
// other channels are in the seven lanes that differ in the low three bits.
template <int CPL>
__device__ __forceinline__ void quantise(const uint32_t (&x)[CPL / 2], uint32_t (&codes)[CPL / 8], __half& s, __half& o) {
  // NaN-propagating, so that one NaN anywhere shows in both
  __half2 lo2 = h2(x[0]), hi2 = lo2;
#pragma unroll
  for (int i = 1; i < CPL / 2; ++i) {
    lo2 = __hmin2_nan(lo2, h2(x[i]));
    hi2 = __hmax2_nan(hi2, h2(x[i]));
  }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    lo2 = __hmin2_nan(lo2, h2(__shfl_xor_sync(0xffffffffu, bits(lo2), m)));
    hi2 = __hmax2_nan(hi2, h2(__shfl_xor_sync(0xffffffffu, bits(hi2), m)));
  }
  const __half lo_h = __hmin_nan(__low2half(lo2), __high2half(lo2)), hi_h = __hmax_nan(__low2half(hi2), __high2half(hi2));
  const float lo = __half2float(lo_h), hi = __half2float(hi_h);
  s = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
  const float sf = __half2float(s);
  o = __float2half_rn(__fmaf_rn(8.0f, sf, lo));
  const float of = __half2float(o);
  // x / s correctly rounded, with one reciprocal for the vector: Markstein's
  // theorem (y the rounded reciprocal, q = x y, q + (x - q s) y)
  const float y = __frcp_rn(sf);
#pragma unroll
  for (int w = 0; w < CPL / 8; ++w) codes[w] = 0;
  if (sf > 0.f) {
#pragma unroll
    for (int i = 0; i < CPL; ++i) {
      const float xi = i & 1 ? __high2float(h2(x[i / 2])) : __low2float(h2(x[i / 2]));
      const float d = __fsub_rn(xi, of);
      const float q0 = __fmul_rn(d, y);
      const float q = __fmaf_rn(__fmaf_rn(-q0, sf, d), y, q0);
      // to an integer, ties to even: the low bits of 1.5 * 2^23 + 8 + q
      const float r = __fadd_rn(fminf(fmaxf(q, -8.f), 7.f), 12582920.f);
      codes[i / 8] |= (__float_as_uint(r) & 15u) << (4 * (i & 7));
    }
  } else {
#pragma unroll
    for (int w = 0; w < CPL / 8; ++w) codes[w] = 0x88888888u;
  }
  if (!(fabsf(lo) <= 65504.f && fabsf(hi) <= 65504.f)) {  // the whole vector reads back as NaN
    s = o = __ushort_as_half(0x7FFF);
#pragma unroll
    for (int w = 0; w < CPL / 8; ++w) codes[w] = 0u;
  }
}

// Codes -> the fp16 values they stand for: s (c - 8) + o in fp32 (c - 8 and its
// product with s are exact), rounded once.
template <int CPL>
__device__ __forceinline__ void dequantise(const uint32_t (&codes)[CPL / 8], uint32_t params, uint32_t (&x)[CPL / 2]) {
  const float2 so = __half22float2(h2(params));
#pragma unroll
  for (int i = 0; i < CPL / 2; ++i) {
    const uint32_t w = codes[i / 4] >> (8 * (i & 3));
    x[i] = bits(__floats2half2_rn(__fmaf_rn(so.x, (float)(int)(w & 15u) - 8.f, so.y),
                                  __fmaf_rn(so.x, (float)(int)((w >> 4) & 15u) - 8.f, so.y)));
  }
}

template <int N>
__device__ __forceinline__ void load_vec(const void* at, uint32_t (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(at)[i];
    x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
  }
}
template <int N>
__device__ __forceinline__ void store_vec(void* at, const uint32_t (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<uint4*>(at)[i] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}

// A token's values into its granule (place i; base nullptr for none), by all lanes of a warp whose four
// groups of eight hold a token each: lane g of a group has channels g D/8 .. + D/8 - 1.
template <int D>
__device__ __forceinline__ void put_values(uint8_t* base, int i, const uint32_t (&vc)[D / 64], int lane) {
  constexpr int CW = D / 32;  // words of a lane's values (paired with another token's)
  const int g = lane & 7, mine = lane >> 3;
  // the token that shares this one's words of values, if it is in this warp: the
  // even one writes the first half of them, the odd one the second
  const int other = (lane + (i & 1 ? -8 : 8)) & 31;
  const bool wraps = i & 1 ? mine == 0 : mine == kTokens - 1;
  const unsigned long long there =
      __shfl_sync(0xffffffffu, base ? (unsigned long long)(uintptr_t)base + i : 0ull, other);
  const bool pair = base && !wraps && there == ((unsigned long long)(uintptr_t)base + i + (i & 1 ? -1 : 1));
  // 16-bit pieces of this token: piece w is channels 4w .. 4w + 3
  uint32_t give, take;
  if constexpr (D == 128) {
    give = i & 1 ? vc[0] : vc[1];
    take = __shfl_sync(0xffffffffu, give, other);
  } else {
    give = vc[0];
    take = __shfl_sync(0xffffffffu, give, other);
  }
  if (!base) return;
  uint8_t* vrow = base + 8 * D + (i >> 3) * (4 * D) + (4 * g + ((i & 7) >> 1)) * (D / 8);
  if constexpr (D == 128) {
    if (pair) {
      // even: pieces 0, 1 of both tokens; odd: pieces 2, 3
      const uint32_t even = i & 1 ? take : vc[0], odd = i & 1 ? vc[1] : take;
      *reinterpret_cast<uint2*>(vrow + (i & 1 ? 8 : 0)) =
          make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
    } else {
#pragma unroll
      for (int w = 0; w < CW; ++w)
        *reinterpret_cast<uint16_t*>(vrow + 4 * w + 2 * (i & 1)) = (uint16_t)(vc[w / 2] >> (16 * (w & 1)));
    }
  } else {
    if (pair) {
      const uint32_t even = i & 1 ? take : vc[0], odd = i & 1 ? vc[0] : take;
      *reinterpret_cast<uint32_t*>(vrow + (i & 1 ? 4 : 0)) = __byte_perm(even, odd, i & 1 ? 0x7632 : 0x5410);
    } else {
#pragma unroll
      for (int w = 0; w < CW; ++w)
        *reinterpret_cast<uint16_t*>(vrow + 4 * w + 2 * (i & 1)) = (uint16_t)(vc[0] >> (16 * w));
    }
  }
}

// kAppend: quantise k, v into the cache; else dequantise the cache into k, v.
template <int D, bool kAppend>
__global__ void __launch_bounds__(kKvThreads) kv_copy_kernel(const KvParams p, __half* k, __half* v, long long k_ts,
                                                             long long k_hs, long long v_ts, long long v_hs) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  constexpr int CPL = D / 8;  // channels per lane
  const int lane = threadIdx.x & 31, g = lane & 7, mine = lane >> 3;
  const long long warp = (long long)blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  const int h = (int)(warp % p.hkv);
  const long long tile = warp / p.hkv;
  const bool live = tile * kTokens + mine < p.T;
  const int t = live ? (int)(tile * kTokens) + mine : 0;
  __half* kp = k + t * k_ts + h * k_hs + g * CPL;
  __half* vp = v + t * v_ts + h * v_hs + g * CPL;
  int i = 0;
  if constexpr (kAppend) {
    uint32_t kx[CPL / 2], vx[CPL / 2];
#pragma unroll
    for (int j = 0; j < CPL / 2; ++j) kx[j] = vx[j] = 0u;
    if (live) {
      load_vec(kp, kx);
      load_vec(vp, vx);
    }
    uint8_t* base = live ? kv_place<D>(p, t, h, &i) : nullptr;
    uint32_t kc[CPL / 8], vc[CPL / 8];
    __half ks, ko, vs, vo;
    quantise<CPL>(kx, kc, ks, ko);
    quantise<CPL>(vx, vc, vs, vo);
    put_values<D>(base, i, vc, lane);
    if (!base) return;
    if constexpr (D == 128)
      *reinterpret_cast<uint2*>(base + i * (D / 2) + g * (CPL / 2)) = make_uint2(kc[0], kc[1]);
    else
      *reinterpret_cast<uint32_t*>(base + i * (D / 2) + g * (CPL / 2)) = kc[0];
    if (g == 0) *reinterpret_cast<uint2*>(base + 16 * D + 8 * i) = make_uint2(pair_bits(ks, ko), pair_bits(vs, vo));
  } else {
    const uint8_t* base = live ? kv_place<D>(p, t, h, &i) : nullptr;
    if (!base) return;
    const uint8_t* vrow = base + 8 * D + (i >> 3) * (4 * D) + (4 * g + ((i & 7) >> 1)) * (D / 8);
    uint32_t kc[CPL / 8], vc[CPL / 8], x[CPL / 2];
    const uint32_t pick = i & 1 ? 0x7632 : 0x5410;
    if constexpr (D == 128) {
      const uint2 kw = *reinterpret_cast<const uint2*>(base + i * (D / 2) + g * (CPL / 2));
      const uint4 vw = *reinterpret_cast<const uint4*>(vrow);
      kc[0] = kw.x;
      kc[1] = kw.y;
      vc[0] = __byte_perm(vw.x, vw.y, pick);
      vc[1] = __byte_perm(vw.z, vw.w, pick);
    } else {
      kc[0] = *reinterpret_cast<const uint32_t*>(base + i * (D / 2) + g * (CPL / 2));
      const uint2 vw = *reinterpret_cast<const uint2*>(vrow);
      vc[0] = __byte_perm(vw.x, vw.y, pick);
    }
    const uint2 pr = *reinterpret_cast<const uint2*>(base + 16 * D + 8 * i);
    dequantise<CPL>(kc, pr.x, x);
    store_vec(kp, x);
    dequantise<CPL>(vc, pr.y, x);
    store_vec(vp, x);
  }
}

template <int D, bool kAppend>
cudaError_t launch_copy(const KvParams& p, uint16_t* k, uint16_t* v, const long long (&st)[4], cudaStream_t stream) {
  const long long warps = ((long long)p.T + kTokens - 1) / kTokens * p.hkv, per = kKvThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)((warps + per - 1) / per));
  cfg.blockDim = dim3(kKvThreads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_copy_kernel<D, kAppend>, p, reinterpret_cast<__half*>(k),
                            reinterpret_cast<__half*>(v), st[0], st[1], st[2], st[3]);
}

// ---- rotary positions and append --------------------------------------------------------------
// (x1, x2) -> (x1 c - x2 s, x2 c + x1 s) for the rot / 2 pairs of the first rot channels, (c, s) the table's
// entry for the pair at the position of its axis: products and sums rounded to fp32 one by one, the
// result to fp16.  Queries go to q_out; keys, and values as they are, into the cache like above.
//
// Bound: the stream, 4 D bytes a query head, 4 D + 2 (D/2 + 4) a key head and token.  The work is steps: four
// tokens like above, eight lanes each, and 1 KB of each: four query heads of 128 channels, or two key heads
// with their values.  Every warp takes an equal run of all steps, in the order of the tokens: what these need
// (their request, place, positions, cosines and sines, a chain of loads) is found once for the steps of the
// same tokens, under the first vectors' loads, and kept in registers.  A lane holds two chunks of D/16
// channels, such that both channels of its pairs are its own: chunks g and g + rot/2 of the rotated ones, two
// neighbours of the rest.
// Measured: 9880 tokens, 32 heads on 8 of 128 channels, three axes, 40.9 us, 5.3 TB/s (79% of the card's copy
// rate; the append alone takes 15.2), 44.0 where the axes of neighbouring pairs differ; 208 tokens, 64 heads on 8, 6.0 us.
template <int D>
constexpr int kVectors = 512 / D;  // together
constexpr int kRopeCtas = 3;  // of an SM

template <int N>  // 4-byte words
__device__ __forceinline__ void load_chunk(const uint16_t* at, uint32_t* x) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    x[0] = v.x; x[1] = v.y;
  }
}
template <int N>
__device__ __forceinline__ void store_chunk(uint16_t* at, const uint32_t* x) {
  if constexpr (N == 4) *reinterpret_cast<uint4*>(at) = make_uint4(x[0], x[1], x[2], x[3]);
  else *reinterpret_cast<uint2*>(at) = make_uint2(x[0], x[1]);
}

__device__ __forceinline__ void rotate(float& x1, float& x2, float2 cs) {
  const float a = x1, b = x2;
  x1 = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  x2 = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// x: a lane's two chunks, CH / 2 words each; cs: of its CH pairs.
template <int CH, bool kInterleaved>
__device__ __forceinline__ void rotate_chunks(uint32_t (&x)[CH], const float2 (&cs)[CH]) {
  if constexpr (kInterleaved) {
#pragma unroll
    for (int w = 0; w < CH; ++w) {
      float2 f = __half22float2(h2(x[w]));
      rotate(f.x, f.y, cs[w]);
      x[w] = bits(__floats2half2_rn(f.x, f.y));
    }
  } else {
#pragma unroll
    for (int w = 0; w < CH / 2; ++w) {
      float2 f = __half22float2(h2(x[w])), s = __half22float2(h2(x[CH / 2 + w]));
      rotate(f.x, s.x, cs[2 * w]);
      rotate(f.y, s.y, cs[2 * w + 1]);
      x[w] = bits(__floats2half2_rn(f.x, f.y));
      x[CH / 2 + w] = bits(__floats2half2_rn(s.x, s.y));
    }
  }
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kKvThreads, kRopeCtas) kv_rope_append_kernel(const KvRopeParams p) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  constexpr int CH = D / 16;  // channels of a chunk, pairs of a lane
  constexpr int kVec = kVectors<D>;
  const int lane = threadIdx.x & 31, g = lane & 7, mine = lane >> 3;
  const int q_steps = (p.heads + kVec - 1) / kVec, steps = q_steps + (2 * p.kv.hkv + kVec - 1) / kVec;
  const long long all = ((long long)p.kv.T + kTokens - 1) / kTokens * steps;
  const long long warp = (long long)blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
  if (warp >= p.warps) return;
  long long begin, end, tile;
  if (all * p.warps < (1ll << 32)) {  // (64-bit divisions are long sequences)
    begin = (uint32_t)(warp * all) / (uint32_t)p.warps;
    end = (uint32_t)((warp + 1) * all) / (uint32_t)p.warps;
    tile = (uint32_t)begin / (uint32_t)steps;
  } else {
    begin = stripe_begin(warp, all, p.warps);
    end = stripe_begin(warp + 1, all, p.warps);
    tile = begin / steps;
  }
  int step = (int)(begin - tile * steps);

  const int half = p.rot / (2 * CH);  // chunks that hold the pairs' first channels (or half of the pairs)
  const bool rotated = g < half;
  const int ca = (rotated ? g : 2 * half + 2 * (g - half)) * CH, cb = rotated ? ca + half * CH : ca + CH;
  int t = 0;
  bool live = false, fresh = true;  // whether there is a token; whether its places and angles are to be found
  bool mine_ok = false;
  uint8_t* base = nullptr;  // the token's granule of key head 0
  int in = 0;
  float2 cs[CH];
  for (long long at = begin; at < end; ++at) {
    if (fresh) {
      live = tile * kTokens + mine < p.kv.T;
      t = live ? (int)(tile * kTokens) + mine : 0;
    }
    const uint16_t *q = p.q + t * p.q_ts, *k = p.k + t * p.k_ts, *v = p.v + t * p.v_ts + g * (D / 8);
    const bool keys = step >= q_steps;
    const int h = keys ? (step - q_steps) * (kVec / 2) : step * kVec;
    const int count = min(kVec, keys ? 2 * (p.kv.hkv - h) : p.heads - h);
    uint32_t x[kVec][CH];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
      for (int w = 0; w < CH; ++w) x[i][w] = 0u;
      if (!live || i >= count) continue;
      if (keys && (i & 1)) {
        const uint16_t* from = v + (h + i / 2) * p.v_hs;
        load_chunk<CH / 2>(from, x[i]);
        load_chunk<CH / 2>(from + CH, x[i] + CH / 2);
      } else {
        const uint16_t* from = keys ? k + (h + i / 2) * p.k_hs : q + (h + i) * p.q_hs;
        load_chunk<CH / 2>(from + ca, x[i]);
        load_chunk<CH / 2>(from + cb, x[i] + CH / 2);
      }
    }
    if (fresh) {
      fresh = false;
      const int b = kv_owner(p.kv, t);
      const KvSeq s = kv_seq(p.kv, b, true);
      mine_ok = live && t >= s.q0 && t < s.q0 + s.nq;
      int pos[kRopeAxes];
#pragma unroll
      for (int a = 0; a < kRopeAxes; ++a) {
        pos[a] = 0;
        if (a < p.axes && mine_ok) pos[a] = p.positions[(long long)a * p.kv.T + t];
      }
      bool bad = false;
#pragma unroll
      for (int a = 0; a < kRopeAxes; ++a) bad = bad || (uint32_t)pos[a] >= (uint32_t)p.table_rows;
      if (bad) {
        if (g == 0) kv_fail(p.kv, kKvSitePosition);
        mine_ok = false;
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) cs[i] = make_float2(1.f, 0.f);
      if (mine_ok && rotated) {
        auto entry = [&](int pair) {
          const int axis = (int)(p.axis[pair >> 5] >> (2 * (pair & 31))) & 3;
          const int at = axis == 0 ? pos[0] : axis == 1 ? pos[1] : axis == 2 ? pos[2] : pos[3];
          return reinterpret_cast<const float2*>(p.table) + (long long)at * (p.rot / 2) + pair;
        };
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int pair0 = kInterleaved ? (part ? cb : ca) / 2 : ca + part * (CH / 2);
          if (p.grouped) {  // CH / 2 pairs lie together
            const float4* from = reinterpret_cast<const float4*>(entry(pair0));
#pragma unroll
            for (int i = 0; i < CH / 4; ++i) {
              const float4 e = from[i];
              cs[part * (CH / 2) + 2 * i] = make_float2(e.x, e.y);
              cs[part * (CH / 2) + 2 * i + 1] = make_float2(e.z, e.w);
            }
          } else {
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) cs[part * (CH / 2) + i] = *entry(pair0 + i);
          }
        }
      }
      base = nullptr;
      if (mine_ok && step + (end - at) > q_steps) base = kv_place_of<D>(p.kv, t, b, s, 0, &in);
    }
    if (++step == steps) {
      step = 0;
      ++tile;
      fresh = true;
    }
    if (!keys) {
      if (!mine_ok) continue;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        if (i >= count) break;
        if (rotated) rotate_chunks<CH, kInterleaved>(x[i], cs);
        uint16_t* to = p.q_out + t * p.o_ts + (h + i) * p.o_hs;
        store_chunk<CH / 2>(to + ca, x[i]);
        store_chunk<CH / 2>(to + cb, x[i] + CH / 2);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      if (i >= count) break;  // (the whole warp)
      if (rotated) rotate_chunks<CH, kInterleaved>(x[i], cs);
      uint32_t kc[CH / 4], vc[CH / 4];
      __half ks, ko, vs, vo;
      quantise<2 * CH>(x[i], kc, ks, ko);
      quantise<2 * CH>(x[i + 1], vc, vs, vo);
      uint8_t* to = base ? base + (h + i / 2) * p.kv.head_bytes : nullptr;
      put_values<D>(to, in, vc, lane);
      if (!to) continue;
      uint8_t* krow = to + in * (D / 2);
      if constexpr (D == 128) {
        *reinterpret_cast<uint32_t*>(krow + ca / 2) = kc[0];
        *reinterpret_cast<uint32_t*>(krow + cb / 2) = kc[1];
      } else {
        *reinterpret_cast<uint16_t*>(krow + ca / 2) = (uint16_t)kc[0];
        *reinterpret_cast<uint16_t*>(krow + cb / 2) = (uint16_t)(kc[0] >> 16);
      }
      if (g == 0) *reinterpret_cast<uint2*>(to + 16 * D + 8 * in) = make_uint2(pair_bits(ks, ko), pair_bits(vs, vo));
    }
  }
}

template <int D, bool kInterleaved>
cudaError_t launch_rope(const KvRopeParams& p, int sms, cudaStream_t stream) {
  constexpr int kVec = kVectors<D>;
  const int steps = (p.heads + kVec - 1) / kVec + (2 * p.kv.hkv + kVec - 1) / kVec;
  KvRopeParams f = p;
  // as many warps as are on the card at a time; a step each, up to twice as many (1290 tokens, 32 heads on 8: 14.3
  // against 14.9 us with the read back)
  const long long all = ((long long)p.kv.T + kTokens - 1) / kTokens * steps, full = (long long)sms * kRopeCtas * (kKvThreads / 32);
  f.warps = all <= 2 * full ? all : full;
  constexpr int per = kKvThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)((f.warps + per - 1) / per));
  cfg.blockDim = dim3(kKvThreads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_rope_append_kernel<D, kInterleaved>, f);
}

}  // namespace

cudaError_t launch_kv_rope_append(const KvRopeParams& p, int D, bool interleaved, int sms, cudaStream_t stream) {
  if (D == 128) return interleaved ? launch_rope<128, true>(p, sms, stream) : launch_rope<128, false>(p, sms, stream);
  return interleaved ? launch_rope<64, true>(p, sms, stream) : launch_rope<64, false>(p, sms, stream);
}

cudaError_t launch_kv_append(const KvParams& p, int D, const uint16_t* k, const uint16_t* v, const long long (&st)[4],
                             cudaStream_t stream) {
  uint16_t *kk = const_cast<uint16_t*>(k), *vv = const_cast<uint16_t*>(v);
  return D == 128 ? launch_copy<128, true>(p, kk, vv, st, stream) : launch_copy<64, true>(p, kk, vv, st, stream);
}

cudaError_t launch_kv_read(const KvParams& p, int D, uint16_t* k, uint16_t* v, const long long (&st)[4],
                           cudaStream_t stream) {
  return D == 128 ? launch_copy<128, false>(p, k, v, st, stream) : launch_copy<64, false>(p, k, v, st, stream);
}

}  // namespace w4a16
