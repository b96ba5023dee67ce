// kv_prefill.cu -- causal attention of many new tokens of a request (a prompt, or
// the next part of one) over the 4-bit paged cache, on tcgen05.
//
// Bound: the two products, 4 D operations per pair of a query row and a token
// it sees, on the tensor cores; beside them one exponential and about ten other
// instructions per pair on the fp32 pipes, and the dequantisation of every
// block once per CTA that reads it.
//   * A CTA (one per SM) owns two tiles of 128 query rows of one key head (the
//     query heads that share it, for consecutive tokens) and passes over the
//     tokens in blocks of 64, dequantised once for both.  The tiles take turns:
//     one's softmax runs under the other's products.
//   * Q stays in shared memory as the A operand of S = Q K^T; S has two places in
//     tensor memory, so that the next block's scores are there when a block's
//     softmax is done; P replaces S as the A operand of O += P V; O stays in
//     tensor memory.
//   * Operands are the codes less 8, exact in fp16; the scales and offsets of
//     keys enter the fp32 scores, those of values P and an fp32 sum per row
//     (kv.cuh has the algebra).  What is rounded is p_t s_t, once, to fp16.
//   * Eight warps own the rows, one per thread; four
//     dequantise the next block into 128-byte-swizzled shared memory; one
//     issues the products.  Channels within groups of eight, and tokens within a
//     block, are in the order in which the codes unpack, in both operands alike.
//   * A row's reference R is chosen so that p_t s_t starts at 2^6 at most; it is
//     only moved, and O rescaled, when some p_t s_t would pass 2^14.
#include <type_traits>

#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kUnset = -1e30f;   // a row's reference before it has seen a token
constexpr float kMost = 16384.f;   // 2^14
constexpr int kTile = 128, kTiles = 2, kRows = kTile * kTiles;  // query rows of a tile and of a CTA
constexpr int kBlock = 64;         // tokens of a block
constexpr int kTileWarps = 4, kSoftmaxWarps = kTiles * kTileWarps, kDequantWarps = 4;
constexpr int kThreadsP = (kSoftmaxWarps + kDequantWarps + 1) * 32;
constexpr int kTmem = 512, kTileCols = kTmem / kTiles;  // columns, and of a tile

struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 dup(float v) { return {v, v}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("{\n\t.reg .b64 ta, tb, tc, td;\n\tmov.b64 ta, {%2, %3};\n\tmov.b64 tb, {%4, %5};\n\tmov.b64 tc, {%6, %7};\n\t"
      "fma.rn.f32x2 td, ta, tb, tc;\n\tmov.b64 {%0, %1}, td;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 ta, tb, td;\n\tmov.b64 ta, {%2, %3};\n\tmov.b64 tb, {%4, %5};\n\t"
      "mul.rn.f32x2 td, ta, tb;\n\tmov.b64 {%0, %1}, td;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 ta, tb, td;\n\tmov.b64 ta, {%2, %3};\n\tmov.b64 tb, {%4, %5};\n\t"
      "add.rn.f32x2 td, ta, tb;\n\tmov.b64 {%0, %1}, td;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<__half2*>(&v)); }

#define W4A16_R32(X)                                                                                                  \
  X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13), X(14), X(15), X(16), X(17), \
      X(18), X(19), X(20), X(21), X(22), X(23), X(24), X(25), X(26), X(27), X(28), X(29), X(30), X(31)
#define W4A16_PLACES32                                                                                             \
  "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, " \
  "%24, %25, %26, %27, %28, %29, %30, %31"

// 32 columns of this thread's lane (32 lanes x 32 bits, 32 repetitions).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
#define W4A16_OUT(i) "=r"(v[i])
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {" W4A16_PLACES32 "}, [%32];"
               : W4A16_R32(W4A16_OUT)
               : "r"(taddr)
               : "memory");
#undef W4A16_OUT
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
#define W4A16_IN(i) "r"(v[i])
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" W4A16_PLACES32 "};" ::W4A16_R32(W4A16_IN), "r"(taddr)
               : "memory");
#undef W4A16_IN
}

// One word of 8 codes -> c - 8 of its nibbles as fp16 pairs, exact: (0, 4),
// (2, 6), (1, 5), (3, 7).  0x6400 | c is 1024 + c, 0x6400 | 16 c is 1024 + 16 c.
__device__ __forceinline__ uint4 unpack8(uint32_t w) {
  uint4 r;
  asm("{\n\t.reg .b32 h, t0, t1, t2, t3;\n\t"
      "shr.u32 h, %4, 8;\n\t"
      "lop3.b32 t0, %4, 0x000F000F, 0x64006400, 0xEA;\n\t"
      "lop3.b32 t1, h, 0x000F000F, 0x64006400, 0xEA;\n\t"
      "lop3.b32 t2, %4, 0x00F000F0, 0x64006400, 0xEA;\n\t"
      "lop3.b32 t3, h, 0x00F000F0, 0x64006400, 0xEA;\n\t"
      "sub.rn.f16x2 %0, t0, %5;\n\t"
      "sub.rn.f16x2 %1, t1, %5;\n\t"
      "fma.rn.f16x2 %2, t2, %6, %7;\n\t"
      "fma.rn.f16x2 %3, t3, %6, %7;\n\t}"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(w), "r"(0x64086408u), "r"(0x2C002C00u), "r"(0xD480D480u));
  return r;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc], kind::f16, issued by an elected lane.
__device__ __forceinline__ void mma_f16_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  }
}

template <int D>
struct ShapeP {
  static constexpr int kK = kBlock * D * 2, kV = D * kBlock * 2;  // bytes of a block's operands
  static constexpr int kPar = kBlock * 16;                        // and of its scales and offsets
  static constexpr int kStages = 3;                              // blocks of operands
  static constexpr int kRaw = 4 * kv_granule_bytes(D);            // a block as it lies in the cache
  static constexpr int kRing = 4;                                 // of them in flight
  static constexpr int kQ = kTile * D * 2;                        // Q of a tile
  static constexpr int kOffV = kStages * kK, kOffQ = kOffV + kStages * kV, kOffPar = kOffQ + kTiles * kQ,
                       kOffRaw = kOffPar + kStages * kPar;
  static constexpr int kSmem = 1024 + kOffRaw + kRing * kRaw;     // alignment slack first
  static_assert(D + 2 * kBlock <= kTileCols, "O and two S of a tile");
  static constexpr int kColO = 0, kColS = D;                      // columns of a tile; P is in S's place
};

struct CtrlP {
  uint64_t kv_full[3], kv_empty[3], raw_full[4], raw_empty[4], s_full[kTiles][2], p_full[kTiles][2], pv_done[kTiles], q_full,
      o_full, drain;
  uint32_t tmem;
  int abort;
  int b, local;
  KvSeq seq;
  alignas(16) float vmax[3][4];  // largest value scale of each granule of a block
};

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1) kv_prefill_kernel(const KvAttnParams p) {
  using Sh = ShapeP<D>;
  constexpr int CW = D / 32, GR = kv_granule_bytes(D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ CtrlP ctrl;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;  // the swizzle's atoms are 1024 bytes
  float* const par0 = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)) + Sh::kOffPar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](uint64_t& b) { return smem_addr(&b); };

  if (tid == 0) {
    for (int s = 0; s < Sh::kStages; ++s) {
      mbar_init(bar(ctrl.kv_full[s]), kDequantWarps);
      mbar_init(bar(ctrl.kv_empty[s]), 1);
    }
    for (int s = 0; s < Sh::kRing; ++s) {
      mbar_init(bar(ctrl.raw_full[s]), 1);
      mbar_init(bar(ctrl.raw_empty[s]), kDequantWarps);
    }
    for (int t = 0; t < kTiles; ++t) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(bar(ctrl.s_full[t][s]), 1);
        mbar_init(bar(ctrl.p_full[t][s]), kTileWarps);
      }
      mbar_init(bar(ctrl.pv_done[t]), 1);
    }
    mbar_init(bar(ctrl.q_full), kSoftmaxWarps);
    mbar_init(bar(ctrl.o_full), 1);
    mbar_init(bar(ctrl.drain), 1);
    ctrl.abort = 0;
    fence_mbarrier_init();
    griddep_launch_dependents();
  }
  kv_prefetch_plan(p.kv, (long long)blockIdx.x * kThreadsP + tid);
  griddep_wait();
  // ---- this CTA's rows: the requests' tiles in order, the last (longest) tile first ------
  if (warp == 0) {
    long long left = blockIdx.x;
    int b = -1;
    KvSeq mine{0, 0, 0};
    for (int b0 = 0; b0 < p.kv.B && b < 0; b0 += 32) {
      KvSeq s{0, 0, 0};
      long long n = 0;
      if (b0 + lane < p.kv.B) {
        s = kv_seq(p.kv, b0 + lane, blockIdx.x == 0);
        if (s.nq > s.len && blockIdx.x == 0) kv_fail(p.kv, kKvSiteLen);
        const long long rows = (long long)s.nq * p.group;
        if (rows > p.min_rows) n = (rows + kRows - 1) / kRows * p.kv.hkv;
      }
      long long upto = n;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, m);
        if (lane >= m) upto += o;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, left < upto);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        left -= __shfl_sync(0xffffffffu, upto - n, src);
        mine.q0 = __shfl_sync(0xffffffffu, s.q0, src);
        mine.nq = __shfl_sync(0xffffffffu, s.nq, src);
        mine.len = __shfl_sync(0xffffffffu, s.len, src);
      } else {
        left -= __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    if (lane == 0) {
      ctrl.b = b;
      ctrl.local = (int)left;
      ctrl.seq = mine;
    }
  }
  __syncthreads();
  const int b = ctrl.b;
  if (b < 0) return;
  if (warp == kSoftmaxWarps + kDequantWarps) {
    tmem_alloc(smem_addr(&ctrl.tmem), kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl.tmem;
  const KvSeq seq = ctrl.seq;
  const WaitCtx wc{&ctrl.abort, p.kv.status, p.timeout_ns};

  const int rows = seq.nq * p.group, tiles = (rows + kRows - 1) / kRows;
  const int h = ctrl.local % p.kv.hkv, row0 = (tiles - 1 - ctrl.local / p.kv.hkv) * kRows;
  const int first = seq.len - seq.nq;  // position of the first new token
  // per tile: tokens any row sees [any_lo, any_hi), tokens every row sees [all_lo,
  // all_hi), and the blocks of the former [from, to)
  int all_lo[kTiles], all_hi[kTiles], from[kTiles], to[kTiles];
  int blk0 = 0x7FFFFFFF, end = 0;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int r0 = row0 + t * kTile, r1 = min(rows, r0 + kTile) - 1;  // first and last row
    const int i0 = r0 / p.group, i1 = r1 / p.group;
    const int any_lo = p.window > 0 ? max(0, first + i0 - p.window + 1) : 0, any_hi = first + i1 + 1;
    all_lo[t] = p.window > 0 ? first + i1 - p.window + 1 : 0;
    all_hi[t] = first + i0 + 1;
    from[t] = any_lo / kBlock;
    to[t] = r0 < rows && any_hi > 0 ? (any_hi + kBlock - 1) / kBlock : from[t];
    if (to[t] > from[t]) {
      blk0 = min(blk0, from[t]);
      end = max(end, to[t]);
    }
  }
  const int n = end > 0 ? end - blk0 : 0;  // blocks of the CTA; 0 where no row sees anything

  if (warp < kSoftmaxWarps) {
    // ================= softmax: a query row per thread =================
    const int tile = warp / kTileWarps;
    const int row = row0 + warp * 32 + lane;
    const bool live = row < rows;
    const int i = live ? row / p.group : 0;
    const int head = h * p.group + (live ? row - i * p.group : 0);
    const int pos = first + i;
    const int hi = live ? pos + 1 : 0, lo = p.window > 0 ? pos - p.window + 1 : 0;  // tokens seen
    const uint32_t lanes = tmem + (uint32_t)(tile * kTileCols) + ((uint32_t)((warp % kTileWarps) * 32) << 16);

    // Q to shared memory, channels in the codes' order; the row's sum
    float qsum = 0.f;
    {
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(seq.q0 + i) * p.q_ts + (long long)head * p.q_hs);
      const int r = row - row0 - tile * kTile;
      const uint32_t qt = base + Sh::kOffQ + tile * Sh::kQ + r * 128;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const uint4 v = live ? src[j] : make_uint4(0u, 0u, 0u, 0u);
        const float2 a = unpack(v.x), bb = unpack(v.y), cc = unpack(v.z), dd = unpack(v.w);
        qsum += ((a.x + a.y) + (bb.x + bb.y)) + ((cc.x + cc.y) + (dd.x + dd.y));
        sts128(qt + (j / 8) * (kTile * 128) + (((j & 7) ^ (r & 7)) << 4),
               make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                          __byte_perm(v.y, v.w, 0x7632)));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ctrl.q_full));
    }
    const F2 qs = dup(qsum);

    float R = live ? kUnset : 0.f;
    F2 l = dup(0.f), pz = dup(0.f);
    bool ok = true;
    const int my_from = tile ? from[1] : from[0], my_n = (tile ? to[1] : to[0]) - my_from;
    const int my_all_lo = tile ? all_lo[1] : all_lo[0], my_all_hi = tile ? all_hi[1] : all_hi[0];
    int stage = my_n > 0 ? (my_from - blk0) % Sh::kStages : 0;
    for (int j = 0; j < my_n; ++j) {
      const int t0 = (my_from + j) * kBlock;
      const uint32_t s_col = lanes + Sh::kColS + (j & 1) * kBlock;
      if (!wait_warp(bar(ctrl.s_full[tile][j & 1]), (uint32_t)((j >> 1) & 1), wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* par = reinterpret_cast<const float4*>(par0 + stage * (Sh::kPar / 4));
      const bool full = t0 >= my_all_lo && t0 + kBlock <= my_all_hi;
      uint32_t P[32];
      F2 lt, pzt;
      float over;
      // one pass over the block's scores; Masked: some row does not see all of it.  A
      // second one where a reference had to be moved.
      auto pass = [&](auto masked) {
        using Masked = decltype(masked);
        lt = pzt = dup(0.f);
        over = 0.f;
        const F2 nr = dup(-R);
        uint32_t sc[2][32];
        tmem_ld32(s_col, sc[0]);
        tmem_wait_ld();
        tmem_ld32(s_col + 32, sc[1]);  // under the first half's arithmetic
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // 32 tokens
          if (half) tmem_wait_ld();
          uint32_t(&s)[32] = sc[half];
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            const float4 kp = par[(half * 32 + t)], vp = par[(half * 32 + t) + 1];  // (ks, ks, ko, ko), (vs, vs, vo, vo)
            F2 x = fma2({kp.x, kp.y}, {__uint_as_float(s[t]), __uint_as_float(s[t + 1])}, fma2({kp.z, kp.w}, qs, nr));
            const int at = t0 + half * 32 + t;
            const bool see0 = !Masked::value || (at < hi && at >= lo), see1 = !Masked::value || (at + 1 < hi && at + 1 >= lo);
            if (!see0) x.x = kNegInf;
            if (!see1) x.y = kNegInf;
            const F2 e = {ex2(x.x), ex2(x.y)};
            lt = add2(lt, e);
            F2 y = mul2(e, {vp.x, vp.y});
            F2 z = Masked::value ? mul2(e, {vp.z, vp.w}) : F2{0.f, 0.f};
            if (Masked::value) {  // a token that is masked for this row may have a NaN scale
              if (!see0) y.x = z.x = 0.f;
              if (!see1) y.y = z.y = 0.f;
              pzt = add2(pzt, z);
            } else {
              pzt = fma2(e, {vp.z, vp.w}, pzt);
            }
            over = fmaxf(over, fmaxf(y.x, y.y));
            // token 16 q + 8 hf + 2 c is pair (4 hf + c) * 4 + q of the operand
            const int q = half * 2 + t / 16, hf = (t / 8) & 1, c = (t / 2) & 3;
            P[(4 * hf + c) * 4 + q] = pack(y.x, y.y);
          }
        }
      };
      over = 2.f * kMost;
      for (int attempt = 0; attempt < 2; ++attempt) {
        if (attempt > 0 || !__any_sync(0xffffffffu, R == kUnset)) {
          if (full) pass(std::false_type{});
          else pass(std::true_type{});
        }
        if (attempt > 0 || !__any_sync(0xffffffffu, over > kMost)) break;
        // move the reference of the rows that need it, rescale what they have
        float top = kNegInf;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t s[32];
          tmem_ld32(s_col + half * 32, s);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < 32; t += 2) {
            const float4 kp = par[half * 32 + t];
            const F2 x = fma2({kp.x, kp.y}, {__uint_as_float(s[t]), __uint_as_float(s[t + 1])}, mul2({kp.z, kp.w}, qs));
            const int at = t0 + half * 32 + t;
            if (at < hi && at >= lo) top = fmaxf(top, x.x);
            if (at + 1 < hi && at + 1 >= lo) top = fmaxf(top, x.y);
          }
        }
        const float4 vm = *reinterpret_cast<const float4*>(ctrl.vmax[stage]);
        const float big = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
        const float scale = (float)max((int)(__float_as_uint(big) >> 23) - 126, -30);  // log2 of a power of two above it
        float f = 1.f;
        if (top > kNegInf && over > kMost) {
          const float nr = top + scale - 6.f;
          if (R == kUnset) {
            R = nr;
          } else if (nr > R) {
            f = ex2(R - nr);
            R = nr;
          }
        }
        l = mul2(l, dup(f));
        pz = mul2(pz, dup(f));
        if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
          // once the products of the blocks before are done (this one's follow P)
          if (!wait_warp(bar(ctrl.pv_done[tile]), (uint32_t)((j - 1) & 1), wc)) break;
          tc_fence_after();
#pragma unroll 1
          for (int part = 0; part < D / 32; ++part) {
            uint32_t v[32];
            tmem_ld32(lanes + Sh::kColO + part * 32, v);
            tmem_wait_ld();
#pragma unroll
            for (int t = 0; t < 32; ++t) v[t] = __float_as_uint(__uint_as_float(v[t]) * f);
            tmem_st32(lanes + Sh::kColO + part * 32, v);
          }
          tmem_wait_st();
        }
      }
      l = add2(l, lt);
      pz = add2(pz, pzt);
      tmem_st32(s_col, P);
      tmem_wait_st();
      tc_fence_before();
      if (lane == 0) mbar_arrive(bar(ctrl.p_full[tile][j & 1]));
      if (++stage == Sh::kStages) stage = 0;
    }
    // ---- the rows' results ----
    if (ok && wait_warp(bar(ctrl.o_full), 0, wc)) {
      tc_fence_after();
      const float sum = l.x + l.y, off = pz.x + pz.y;
      const float inv = hi > 0 ? 1.f / sum : 0.f;  // a row that sees no token is zero
      uint16_t* dst = p.out + ((long long)(seq.q0 + i) * p.heads + head) * D;
#pragma unroll 1
      for (int part = 0; part < D / 32; ++part) {
        uint32_t v[32];
        tmem_ld32(lanes + Sh::kColO + part * 32, v);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int t = 0; t < 32; t += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float a = (__uint_as_float(v[t + 2 * k]) + off) * inv, c = (__uint_as_float(v[t + 2 * k + 1]) + off) * inv;
              if (inv == 0.f) a = c = 0.f;
              w[k] = pack(a, c);
            }
            *reinterpret_cast<uint4*>(dst + part * 32 + t) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  } else if (warp < kSoftmaxWarps + kDequantWarps) {
    // ================= dequantisation =================
    const int dw = warp - kSoftmaxWarps, g = lane >> 2, c = lane & 3;
    const int half = dw >> 1, wp = dw & 1;  // this warp's part of the values
    // warp 0 of the four keeps kRing blocks in flight: lane q < 4 copies granule q
    const int* table = p.kv.table + (long long)b * p.kv.max_pages;
    const uint8_t* heads = p.kv.cache + h * p.kv.head_bytes;
    const uint64_t policy = policy_evict_last();  // other CTAs read the same blocks
    const uint32_t raw = base + Sh::kOffRaw;
    int next_page = 0, issued = 0;
    auto look_up = [&]() {
      const int gi = (blk0 + issued) * 4 + lane;
      if (lane < 4 && gi * kGranule < seq.len) next_page = table[kv_div_page(p.kv, gi)];
    };
    auto issue = [&]() {
      const int gi = (blk0 + issued) * 4 + lane, slot = issued % Sh::kRing;
      const bool inside = lane < 4 && gi * kGranule < seq.len;
      const bool there = inside && (uint32_t)next_page < (uint32_t)p.kv.n_pages;
      if (inside && !there) kv_fail(p.kv, kKvSitePage);  // no copy: the results are not valid, and reported
      const int copies = __popc(__ballot_sync(0xffffffffu, there));
      if (lane == 0) mbar_arrive_expect_tx(bar(ctrl.raw_full[slot]), copies * GR);
      __syncwarp();
      if (there && (lane == 0 || !p.whole_blocks))
        bulk_g2s(raw + slot * Sh::kRaw + lane * GR,
                 heads + next_page * p.kv.page_bytes + (gi - kv_div_page(p.kv, gi) * p.kv.page16) * GR,
                 p.whole_blocks ? copies * GR : GR, bar(ctrl.raw_full[slot]), policy);
      if (++issued < n) look_up();
    };
    if (dw == 0) {
      look_up();
      while (issued < min(Sh::kRing, n)) issue();
    }
    const uint8_t* raw_ptr = smem_raw + (base - smem_addr(smem_raw)) + Sh::kOffRaw;
    int j = 0, stage = 0;
    uint32_t ph = 0;
    for (; j < n; ++j) {
      if (!wait_warp(bar(ctrl.raw_full[j % Sh::kRing]), (uint32_t)((j / Sh::kRing) & 1), wc)) break;
      const uint8_t* in = raw_ptr + (j % Sh::kRing) * Sh::kRaw;
      uint32_t k0[CW], k1[CW], vv[4][CW / 2];
      load_words<CW>(in + dw * GR + g * (D / 2) + c * (D / 8), k0);
      load_words<CW>(in + dw * GR + (g + 8) * (D / 2) + c * (D / 8), k1);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        load_words<CW / 2>(in + q * GR + 8 * D + half * (4 * D) + lane * (D / 8) + wp * (D / 16), vv[q]);
      // nothing is taken from tokens that are not written (they may hold anything)
      uint2 pr = make_uint2(0u, 0u);
      if (lane < 16 && ((blk0 + j) * 4 + dw) * kGranule + lane < seq.len)
        pr = *reinterpret_cast<const uint2*>(in + dw * GR + 16 * D + 8 * lane);
      if (!wait_warp(bar(ctrl.kv_empty[stage]), ph ^ 1u, wc)) break;
      const uint32_t kt = base + stage * Sh::kK, vt = base + Sh::kOffV + stage * Sh::kV;
      // keys: row = token, 16-byte unit = 8 channels; lanes with c >= 2 take their words
      // in another order, so that eight lanes write eight different units
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 16 * dw + 8 * e + g;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
          if constexpr (CW == 4) {
            const uint32_t a = e ? k1[w] : k0[w], d = e ? k1[w ^ 2] : k0[w ^ 2];
            const int unit = (c & 1) * 4 + (c & 2 ? w ^ 2 : w);
            sts128(kt + (c >> 1) * (kBlock * 128) + t * 128 + ((unit ^ (t & 7)) << 4), unpack8(c & 2 ? d : a));
          } else {
            sts128(kt + t * 128 + (((c * 2 + w) ^ (t & 7)) << 4), unpack8(e ? k1[w] : k0[w]));
          }
        }
      }
      // values: row = channel, 16-byte unit 4 half + c = the pair of tokens 8 half + 2 c of
      // each granule; odd g take their two words in the other order, for the same reason
#pragma unroll
      for (int w = 0; w < CW / 2; ++w) {
        const int mine = CW == 4 && (g & 1) ? w ^ 1 : w;
        uint4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t a = vv[q][w], d = vv[q][CW == 4 ? w ^ 1 : w];
          x[q] = unpack8(CW == 4 && (g & 1) ? d : a);
        }
        const int ch = g * (D / 8) + 4 * (wp * (CW / 2) + mine), unit = 4 * half + c;
        auto put = [&](int k, uint32_t a, uint32_t b2, uint32_t c2, uint32_t d2) {
          sts128(vt + (ch + k) * 128 + ((unit ^ ((ch + k) & 7)) << 4), make_uint4(a, b2, c2, d2));
        };
        put(0, x[0].x, x[1].x, x[2].x, x[3].x);
        put(2, x[0].y, x[1].y, x[2].y, x[3].y);
        put(1, x[0].z, x[1].z, x[2].z, x[3].z);
        put(3, x[0].w, x[1].w, x[2].w, x[3].w);
      }
      // scales and offsets, by pairs of tokens: (ks, ks, ko, ko, vs, vs, vo, vo), keys' in log2 units
      {
        const float2 kf = unpack(pr.x), vf = unpack(pr.y);
        float big = lane < 16 ? vf.x : 0.f;
        big = big > 0.f ? big : 0.f;  // also of a NaN
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
        if (lane < 16) {
          float* dst = par0 + stage * (Sh::kPar / 4) + (16 * dw + (lane & ~1)) * 4 + (lane & 1);
          dst[0] = kf.x * p.scale_log2;
          dst[2] = kf.y * p.scale_log2;
          dst[4] = vf.x;
          dst[6] = vf.y;
        }
        if (lane == 0) ctrl.vmax[stage][dw] = big;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(ctrl.kv_full[stage]));
        mbar_arrive(bar(ctrl.raw_empty[j % Sh::kRing]));
      }
      // the slot of the block before this one, which the others are done with by now
      if (dw == 0 && j > 0 && issued < n) {
        if (!wait_warp(bar(ctrl.raw_empty[(j - 1) % Sh::kRing]), (uint32_t)(((j - 1) / Sh::kRing) & 1), wc)) {
          ++j;
          break;
        }
        issue();
      }
      if (++stage == Sh::kStages) {
        stage = 0;
        ph ^= 1u;
      }
    }
    // nothing may still be in flight into this CTA's shared memory
    if (dw == 0 && lane == 0)
      for (; j < issued; ++j)
        wait_drain(bar(ctrl.raw_full[j % Sh::kRing]), (uint32_t)((j / Sh::kRing) & 1), wc);
  } else {
    // ================= products =================
    const uint32_t id_s = umma_idesc_f16_f32(kBlock), id_o = umma_idesc_f16_f32(D);
    int stage = 0, next = Sh::kStages > 1 ? 1 : 0;  // of block j and of the one after it
    uint32_t next_ph = 0;
    // S = Q K^T of a tile's i-th block.  The place is free: the P that was there was
    // consumed by a product before, which these follow in order.
    auto scores = [&](int t, int i, int st) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_f16_ss_elect(tmem + t * kTileCols + Sh::kColS + (i & 1) * kBlock,
                         umma_desc_sw128(base + Sh::kOffQ + t * Sh::kQ + (kk / 4) * (kTile * 128)) + (uint64_t)(2 * (kk & 3)),
                         umma_desc_sw128(base + st * Sh::kK + (kk / 4) * (kBlock * 128)) + (uint64_t)(2 * (kk & 3)), id_s,
                         kk > 0);
      mma_commit_elect(bar(ctrl.s_full[t][i & 1]));
    };
    bool ok = wait_warp(bar(ctrl.q_full), 0, wc);
    if (ok && n > 0 && (ok = wait_warp(bar(ctrl.kv_full[0]), 0, wc))) {
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (from[t] == blk0 && to[t] > blk0) scores(t, 0, 0);
    }
    for (int j = 0; ok && j < n; ++j) {
      const int blk = blk0 + j;
      if (j + 1 < n) {  // the next block's scores go before this one's products with V
        if (!(ok = wait_warp(bar(ctrl.kv_full[next]), next_ph, wc))) break;
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
          if (blk + 1 >= from[t] && blk + 1 < to[t]) scores(t, blk + 1 - from[t], next);
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int i = blk - from[t];
        if (!ok || i < 0 || blk >= to[t]) continue;
        if (!(ok = wait_warp(bar(ctrl.p_full[t][i & 1]), (uint32_t)((i >> 1) & 1), wc))) continue;
        tc_fence_after();
        const uint32_t cols = tmem + t * kTileCols;
#pragma unroll
        for (int kk = 0; kk < kBlock / 16; ++kk)
          mma_f16_ts_elect(cols + Sh::kColO, cols + Sh::kColS + (i & 1) * kBlock + kk * 8,
                           umma_desc_sw128(base + Sh::kOffV + stage * Sh::kV) + (uint64_t)(2 * kk), id_o, i > 0 || kk > 0);
        mma_commit_elect(bar(ctrl.pv_done[t]));
      }
      if (!ok) break;
      mma_commit_elect(bar(ctrl.kv_empty[stage]));
      stage = next;
      if (++next == Sh::kStages) {
        next = 0;
        next_ph ^= 1u;
      }
    }
    if (ok) mma_commit_elect(bar(ctrl.o_full));
    mma_commit_elect(bar(ctrl.drain));
    wait_drain(bar(ctrl.drain), 0, wc);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftmaxWarps + kDequantWarps) tmem_dealloc(tmem, kTmem);
}

template <int D>
cudaError_t launch(const KvAttnParams& p, long long grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = ShapeP<D>::kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_prefill_kernel<D>, p);
}

}  // namespace

cudaError_t kv_prefill_set_smem_limit() {
  cudaError_t e = cudaFuncSetAttribute(kv_prefill_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       ShapeP<128>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv_prefill_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, ShapeP<64>::kSmem);
  return e;
}

cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, cudaStream_t stream) {
  // groups of 256 rows: at most one part-filled for each request
  const long long grid = ((long long)p.kv.T * p.group / kRows + p.kv.B) * p.kv.hkv;
  return D == 128 ? launch<128>(p, grid, stream) : launch<64>(p, grid, stream);
}

}  // namespace w4a16
