// kv_cache.cu -- writing new keys and values into the 4-bit paged cache, and
// reading cached values back as fp16.
//
// Both are streams: 4 D bytes of fp16 in (or out) and D + 8 bytes of cache per
// token and head, a handful of operations per channel.
#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr int kKvThreads = 256;

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

// Byte offset in a granule's V part of channels 4 l .. 4 l + 3 of token i.
template <int D>
__device__ __forceinline__ int v_offset(int i, int l) {
  constexpr int kWords = D / 32;  // words of four channels per (g, c)
  const int g = l / kWords, w = l % kWords;
  return (i >> 3) * (4 * D) + (4 * g + ((i & 7) >> 1)) * (D / 8) + 4 * w + 2 * (i & 1);
}

// Four channels of one vector per lane, D/4 lanes together: the codes of the
// lane's channels (16 bits), and the vector's scale and offset.
template <int LG>
__device__ __forceinline__ uint32_t quantise(uint2 raw, __half* s_out, __half* o_out) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&raw.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&raw.y));
  const float x[4] = {a.x, a.y, b.x, b.y};
  float lo = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
  float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  // a NaN or infinity anywhere: x - x is NaN there, and sums keep it
  float bad = (x[0] - x[0]) + (x[1] - x[1]) + (x[2] - x[2]) + (x[3] - x[3]);
#pragma unroll
  for (int m = 1; m < LG; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    bad += __shfl_xor_sync(0xffffffffu, bad, m);
  }
  __half s = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
  const float sf = __half2float(s);
  __half o = __float2half_rn(__fmaf_rn(8.0f, sf, lo));
  const float of = __half2float(o);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float c = sf > 0.f ? rintf(__fdiv_rn(__fsub_rn(x[i], of), sf)) : 0.f;
    c = fminf(fmaxf(c, -8.f), 7.f);
    codes |= (uint32_t)((int)c + 8) << (4 * i);
  }
  if (bad != 0.f) {  // NaN compares unequal: the whole vector reads back as NaN
    s = o = __ushort_as_half(0x7FFF);
    codes = 0;
  }
  *s_out = s;
  *o_out = o;
  return codes;
}

// Four codes (16 bits) -> the fp16 values they stand for: s (c - 8) + o in
// fp32 (c - 8 and its product with s are exact), rounded once.
__device__ __forceinline__ uint2 dequantise(uint32_t codes, float s, float o) {
  __half h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __float2half_rn(__fmaf_rn(s, (float)(int)((codes >> (4 * i)) & 15u) - 8.f, o));
  const __half2 a = __halves2half2(h[0], h[1]), b = __halves2half2(h[2], h[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ uint32_t pair_bits(__half a, __half b) {
  return (uint32_t)__half_as_ushort(a) | ((uint32_t)__half_as_ushort(b) << 16);
}

// kAppend: quantise k, v into the cache; else dequantise the cache into k, v.
template <int D, bool kAppend>
__global__ void __launch_bounds__(kKvThreads) kv_copy_kernel(const KvParams p, __half* k, __half* v, long long k_ts,
                                                             long long k_hs, long long v_ts, long long v_hs) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();
  constexpr int LG = D / 4;  // lanes per vector
  const int l = threadIdx.x % LG;
  const long long item = (long long)blockIdx.x * (kKvThreads / LG) + threadIdx.x / LG;
  const bool live = item < (long long)p.T * p.hkv;
  const int t = live ? (int)(item / p.hkv) : 0;
  const int h = live ? (int)(item - (long long)t * p.hkv) : 0;
  uint2* kp = reinterpret_cast<uint2*>(k + t * k_ts + h * k_hs + 4 * l);
  uint2* vp = reinterpret_cast<uint2*>(v + t * v_ts + h * v_hs + 4 * l);
  int i = 0;
  if (kAppend) {
    // the vectors' loads go out before the look-ups of their place
    const uint2 kr = live ? *kp : make_uint2(0u, 0u), vr = live ? *vp : make_uint2(0u, 0u);
    uint8_t* base = live ? kv_place<D>(p, t, h, &i) : nullptr;
    __half ks, ko, vs, vo;
    const uint32_t kc = quantise<LG>(kr, &ks, &ko);
    const uint32_t vc = quantise<LG>(vr, &vs, &vo);
    if (!base) return;
    *reinterpret_cast<uint16_t*>(base + i * (D / 2) + 2 * l) = (uint16_t)kc;
    *reinterpret_cast<uint16_t*>(base + 8 * D + v_offset<D>(i, l)) = (uint16_t)vc;
    if (l == 0)
      *reinterpret_cast<uint2*>(base + 16 * D + 8 * i) = make_uint2(pair_bits(ks, ko), pair_bits(vs, vo));
  } else {
    const uint8_t* base = live ? kv_place<D>(p, t, h, &i) : nullptr;
    if (!base) return;
    const uint32_t kc = *reinterpret_cast<const uint16_t*>(base + i * (D / 2) + 2 * l);
    const uint32_t vc = *reinterpret_cast<const uint16_t*>(base + 8 * D + v_offset<D>(i, l));
    const uint2 pr = *reinterpret_cast<const uint2*>(base + 16 * D + 8 * i);
    const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&pr.x));
    const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&pr.y));
    *kp = dequantise(kc, kf.x, kf.y);
    *vp = dequantise(vc, vf.x, vf.y);
  }
}

template <int D, bool kAppend>
cudaError_t launch_copy(const KvParams& p, uint16_t* k, uint16_t* v, const long long (&st)[4], cudaStream_t stream) {
  const long long per = kKvThreads / (D / 4), items = (long long)p.T * p.hkv;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)((items + per - 1) / per));
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
