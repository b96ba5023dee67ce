// kv_cache.cu -- writing new keys and values into the 4-bit paged cache, and
// reading cached values back as fp16.
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
#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr int kKvThreads = 256;
constexpr int kTokens = 4;  // of a warp

// Where token t (of all new tokens) of head h lives: its granule, and its
// place in it; nullptr if the inputs give it none.
template <int D>
__device__ __forceinline__ uint8_t* kv_place(const KvParams& p, int t, int h, int* in_granule) {
  // the request that owns token t: the last b with q_start[b] <= t
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const KvSeq s = kv_seq(p, lo, true);
  if (t < s.q0 || t >= s.q0 + s.nq) return nullptr;
  const int pos = s.len - (s.q0 + s.nq - t);
  if (pos < 0) {
    kv_fail(p, kKvSiteLen);
    return nullptr;
  }
  const int g16 = pos >> 4;
  const int pi = kv_div_page(p, g16);
  const int page = p.table[(long long)lo * p.max_pages + pi];
  if (page < 0 || page >= p.n_pages) {
    kv_fail(p, kKvSitePage);
    return nullptr;
  }
  *in_granule = pos & 15;
  return p.cache + page * p.page_bytes + h * p.head_bytes + (long long)(g16 - pi * p.page16) * kv_granule_bytes(D);
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

// kAppend: quantise k, v into the cache; else dequantise the cache into k, v.
template <int D, bool kAppend>
__global__ void __launch_bounds__(kKvThreads) kv_copy_kernel(const KvParams p, __half* k, __half* v, long long k_ts,
                                                             long long k_hs, long long v_ts, long long v_hs) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  constexpr int CPL = D / 8, CW = D / 32;  // channels per lane; words of a lane's values (paired with another token's)
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
      *reinterpret_cast<uint2*>(base + i * (D / 2) + g * (CPL / 2)) = make_uint2(kc[0], kc[1]);
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
      *reinterpret_cast<uint32_t*>(base + i * (D / 2) + g * (CPL / 2)) = kc[0];
      if (pair) {
        const uint32_t even = i & 1 ? take : vc[0], odd = i & 1 ? vc[0] : take;
        *reinterpret_cast<uint32_t*>(vrow + (i & 1 ? 4 : 0)) = __byte_perm(even, odd, i & 1 ? 0x7632 : 0x5410);
      } else {
#pragma unroll
        for (int w = 0; w < CW; ++w)
          *reinterpret_cast<uint16_t*>(vrow + 4 * w + 2 * (i & 1)) = (uint16_t)(vc[0] >> (16 * w));
      }
    }
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

}  // namespace

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
