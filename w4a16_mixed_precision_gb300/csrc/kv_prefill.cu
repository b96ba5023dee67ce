// kv_prefill.cu -- causal attention of many new tokens of a request (a prompt, or
// the next part of one) over the 4-bit paged cache, on tcgen05.
//
// Bound: the two products, 4 D operations per pair of a query row and a token
// it sees, on the tensor cores; beside them one exponential and about ten other
// instructions per pair on the fp32 pipes, and the dequantisation of every
// block once per CTA that reads it.
//   * An item is 256 query rows, two tiles of 128, of one key head (the query heads
//     that share it, for consecutive tokens), which passes over the tokens it
//     sees in blocks of 64, dequantised once for both tiles.  A CTA (one per SM)
//     takes one item, or, where there would be few or long ones, an equal stripe
//     of all items' blocks; the rule is at find_item.  Either is found on the
//     device.  An item that stripes cut is finished by the last of its CTAs to
//     arrive, in stripe order.
//   * Q stays in shared memory as the A operand of S = Q K^T; S has two places in
//     tensor memory, so that the next block's scores are there when a block's
//     softmax is done; P replaces S as the A operand of O += P V; O stays in
//     tensor memory.
//   * Operands are the codes less 8, exact in fp16; the scales and offsets of
//     keys enter the fp32 scores, those of values P and an fp32 sum per row
//     (kv.cuh has the algebra).  What is rounded is p_t s_t, once, to fp16: the error
//     against 64 bits is 2.7 to 3.0e-4 of the result, where the output's own rounding
//     leaves 2.1e-4; a second fp16 number for the rest would double the products with V.
//   * Eight warps own the rows, one per thread; four
//     dequantise the next block into 128-byte-swizzled shared memory; one
//     issues the products.  Channels within groups of eight, and tokens within a
//     block, are in the order in which the codes unpack, in both operands alike.
//   * A row's reference R is chosen so that p_t s_t starts at 2^6 at most; it is
//     only moved, and O rescaled, when some p_t s_t (s_t taken as 2^-30 at least)
//     would pass 2^14.
//
// Measured: 1000 new tokens on 9000, 64 query heads on 8 of 128 channels, 355 us,
// 785 TFLOP/s (40% of the card's bf16 rate); the prompts of 5 requests of 682 to
// 1900 tokens, 32 heads, 184 us, 404 TFLOP/s.  A block of 64 tokens for 256 rows
// takes about 2700 cycles, of which shared memory needs 1950 (Q and K for S, V, the
// dequantised block's writes, scales and offsets), the softmax warps' instructions
// 1650 and the products 1540 (N is 64 for S, and costs nearly what 128 would): no one
// of them is the bound alone.  Short items also pay about 6 us each for their
// start, their first (longer) block and their rows' results.  Tried and slower: one
// tile per CTA (the block dequantised for 128 rows only), S = Q K^T with Q in
// tensor memory, products issued by the softmax warps.
#include <type_traits>

#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kUnset = -1e30f;   // a row's reference before it has seen a token
constexpr float kMost = 16384.f;   // 2^14
constexpr float kLeastScale = 9.313225746154785e-10f;  // 2^-30
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
  uint64_t part_done, verdict;
  uint32_t tmem;
  int abort;
  int last;             // whether this CTA joins the parts of an item
  int by_item;          // whether a CTA takes one whole item
  int start_b, start_h, start_tile, start_x;
  long long sums[16], items[16];  // blocks and items of the requests of each warp
  int longest[16];                // blocks of their longest item
  alignas(16) float vmax[3][4];  // largest value scale of each granule of a block
};

// Blocks that the rows of an item see: [lo, lo + n), one (masked) block where
// they see nothing.
struct Span {
  int lo, n;
};
__device__ __forceinline__ Span item_span(const KvAttnParams& p, const KvSeq& s, int rows, int tile) {
  const int r0 = tile * kRows, r1 = min(rows, r0 + kRows) - 1, first = s.len - s.nq;
  const int lo = p.window > 0 ? max(0, first + kv_div_group(p, r0) - p.window + 1) / kBlock : 0;
  const int hi = (max(0, first + kv_div_group(p, r1) + 1) + kBlock - 1) / kBlock;
  return {lo, max(1, hi - lo)};
}

// Rows of a request, 0 where another launch takes it.
__device__ __forceinline__ int item_rows(const KvAttnParams& p, const KvSeq& s) {
  const int rows = s.nq * p.group;
  return rows > p.min_rows ? rows : 0;
}

// Blocks of all items of a request and one key head, by a warp; and its longest item's.
__device__ __forceinline__ long long request_blocks(const KvAttnParams& p, const KvSeq& s, int* longest) {
  const int rows = item_rows(p, s), tiles = (rows + kRows - 1) / kRows;
  long long sum = 0;
  int most = 0;
  for (int t = threadIdx.x & 31; t < tiles; t += 32) {
    const int n = item_span(p, s, rows, t).n;
    sum += n;
    most = max(most, n);
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, m);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, m));
  }
  *longest = max(*longest, most);
  return sum;
}

// A place in the stripe: block x of an item; items in the order request, key
// head, tile (the last, longest one first).
struct Place {
  int b, h, tile, x;
  int left;            // blocks of the stripe from here on
  KvSeq seq;
  int rows;
  Span span;           // of the item
};

__device__ __forceinline__ void enter_item(const KvAttnParams& p, Place& c) { c.span = item_span(p, c.seq, c.rows, c.tile); }

// One of an item's two tiles, in blocks [from, to) of the piece [blk0, end): those
// that any of its rows sees; and the tokens that all of them see.
struct Half {
  int from, to, all_lo, all_hi;
};
__device__ __forceinline__ Half tile_half(const KvAttnParams& p, const Place& c, int t, int blk0, int end) {
  const int r0 = c.tile * kRows + t * kTile, r1 = min(c.rows, r0 + kTile) - 1, first = c.seq.len - c.seq.nq;
  const int i0 = kv_div_group(p, r0), i1 = kv_div_group(p, r1);
  Half f;
  f.all_lo = p.window > 0 ? first + i1 - p.window + 1 : 0;
  f.all_hi = first + i0 + 1;
  f.from = max(blk0, p.window > 0 ? max(0, first + i0 - p.window + 1) / kBlock : 0);
  f.to = r0 < c.rows ? min(end, (max(0, first + i1 + 1) + kBlock - 1) / kBlock) : f.from;
  if (f.to < f.from) f.to = f.from;
  return f;
}

// Moves on by `by` blocks, to the end of the item at most.
__device__ __forceinline__ void move_on(const KvAttnParams& p, Place& c, int by) {
  c.x += by;
  c.left -= by;
  if (c.x < c.span.n || c.left <= 0) return;
  c.x = 0;
  if (--c.tile < 0) {
    if (++c.h == p.kv.hkv) {
      c.h = 0;
      do {
        if (++c.b >= p.kv.B) {
          c.left = 0;
          return;
        }
        c.seq = kv_seq(p.kv, c.b, false);
        c.rows = item_rows(p, c.seq);
      } while (c.rows == 0);
    }
    c.tile = (c.rows + kRows - 1) / kRows - 1;
  }
  enter_item(p, c);
}

// The blockIdx.x-th item, each request's longest first, by a warp, where the grid has
// a CTA for every item.  But not where stripes are expected to end before the last
// of the items: these end after as many of the longest as an SM takes, or half of one
// after the mean, whichever is less; stripes at the mean (U / S blocks), and what
// starting, publishing and joining parts costs.  Measured with 128 channels, items
// against stripes: 256 items of 16 blocks at most 47 against 77 us, 576 of 24 at most
// 124 against 153, 1264 of 40 at most 325 against 442; 256 of 126 to 141 blocks 389
// against 355, 376 of 94 to 141 506 against 462, 504 of 94 to 125 629 against 573.
// The mean is taken as if a request's items grew evenly.
constexpr int kCutCost = 20, kCutItemCost = 4;  // blocks
__device__ __forceinline__ void find_item(const KvAttnParams& p, CtrlP& ctrl) {
  const int lane = threadIdx.x & 31;
  long long left = blockIdx.x, U = 0, items = 0;
  int longest = 0;
  bool found = false;
  for (int b0 = 0; b0 < p.kv.B; b0 += 32) {
    long long n = 0;
    int tiles = 0;
    if (b0 + lane < p.kv.B) {
      const KvSeq s = kv_seq(p.kv, b0 + lane, blockIdx.x == 0);
      if (s.nq > s.len && blockIdx.x == 0) kv_fail(p.kv, kKvSiteLen);
      const int rows = item_rows(p, s);
      tiles = (rows + kRows - 1) / kRows;
      n = (long long)tiles * p.kv.hkv;
      if (tiles > 0) {
        const int n0 = item_span(p, s, rows, 0).n, n1 = item_span(p, s, rows, tiles - 1).n;
        longest = max(longest, max(n0, n1));
        U += n * (n0 + n1) / 2;
      }
    }
    long long upto = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, m);
      if (lane >= m) upto += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, left < upto);
    if (!found && hit && lane == __ffs(hit) - 1) {
      const int k = (int)(left - (upto - n));
      ctrl.start_b = b0 + lane;
      ctrl.start_h = k % p.kv.hkv;
      ctrl.start_tile = tiles - 1 - k / p.kv.hkv;
      ctrl.start_x = 0;
    }
    found = found || hit;
    const long long all = __shfl_sync(0xffffffffu, upto, 31);
    left -= all;
    items += all;
  }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    U += __shfl_xor_sync(0xffffffffu, U, m);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, m));
  }
  __syncwarp();
  const long long S = p.stripes, mean = U / S;
  const long long whole = min((items + S - 1) / S * longest, mean + longest / 2);
  if (items <= (long long)gridDim.x && whole <= mean + kCutCost + kCutItemCost * items / S) {
    if (lane == 0) ctrl.by_item = 1;
  } else if (lane == 0) {
    ctrl.start_b = -1;
  }
}

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
    mbar_init(bar(ctrl.part_done), kSoftmaxWarps);
    mbar_init(bar(ctrl.verdict), 1);
    mbar_init(bar(ctrl.o_full), 1);
    mbar_init(bar(ctrl.drain), 1);
    ctrl.abort = 0;
    ctrl.by_item = 0;
    ctrl.start_b = -1;
    fence_mbarrier_init();
    griddep_launch_dependents();
  }
  kv_prefetch_plan(p.kv, (long long)blockIdx.x * kThreadsP + tid);
  griddep_wait();
  if (warp == kSoftmaxWarps + kDequantWarps) {
    tmem_alloc(smem_addr(&ctrl.tmem), kTmem);
    tmem_relinquish();
  }
  // ---- this CTA's work: an item, or a stripe of all items ----------------------------------
  const bool many = (int)gridDim.x > p.stripes;
  if (many && warp == 0) find_item(p, ctrl);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl.tmem;
  bool by_item = ctrl.by_item;
  if (by_item && ctrl.start_b < 0) {  // no item for this CTA
    if (warp == kSoftmaxWarps + kDequantWarps) tmem_dealloc(tmem, kTmem);
    return;
  }
  long long U = 0, G = 0, u_begin = 0, u_end = 0;
  if (!by_item) {
    // every warp sums a run of requests; the warp whose run holds the CTA's first block finds it
    constexpr int kWarps = kThreadsP / 32;
    const int per = (p.kv.B + kWarps - 1) / kWarps, b_from = min(warp * per, p.kv.B), b_to = min(b_from + per, p.kv.B);
    long long mine = 0, mine_items = 0;
    int longest = 0;
    for (int b = b_from; b < b_to; ++b) {
      const KvSeq q = kv_seq(p.kv, b, blockIdx.x == 0 && lane == 0);
      if (q.nq > q.len && blockIdx.x == 0 && lane == 0) kv_fail(p.kv, kKvSiteLen);
      mine += p.kv.hkv * request_blocks(p, q, &longest);
      mine_items += (long long)p.kv.hkv * ((item_rows(p, q) + kRows - 1) / kRows);
    }
    if (lane == 0) {
      ctrl.sums[warp] = mine;
      ctrl.items[warp] = mine_items;
      ctrl.longest[warp] = longest;
    }
    __syncthreads();
    long long before = 0, all_items = 0, items_before = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        before = U;
        items_before = all_items;
      }
      U += ctrl.sums[w];
      all_items += ctrl.items[w];
      longest = max(longest, ctrl.longest[w]);
    }
    // no more items than SMs: a CTA each, unless stripes would end before the longest
    by_item = !many && all_items <= (long long)gridDim.x && longest <= U / p.stripes + kCutCost;
    G = by_item ? all_items : min((long long)p.stripes, U);
    const bool works = (long long)blockIdx.x < G;
    if (works && !by_item) {
      u_begin = stripe_begin(blockIdx.x, U, G);
      u_end = stripe_begin(blockIdx.x + 1, U, G);
    }
    const long long at_unit = by_item ? blockIdx.x : u_begin;
    const long long from_unit = by_item ? items_before : before;
    if (works && at_unit >= from_unit && at_unit < from_unit + (by_item ? mine_items : mine)) {
      long long off = at_unit - from_unit;
      for (int b = b_from; b < b_to; ++b) {
        const KvSeq q = kv_seq(p.kv, b, false);
        const int rows = item_rows(p, q), tiles = (rows + kRows - 1) / kRows;
        const long long one = by_item ? tiles : request_blocks(p, q, &longest);
        if (off >= one * p.kv.hkv) {
          off -= one * p.kv.hkv;
          continue;
        }
        const int h = (int)(off / one);
        off -= h * one;
        if (by_item) {
          if (lane == 0) {
            ctrl.start_b = b;
            ctrl.start_h = h;
            ctrl.start_tile = tiles - 1 - (int)off;
            ctrl.start_x = 0;
          }
          break;
        }
        for (int top = tiles - 1; top >= 0; top -= 32) {  // 32 tiles at a time, downwards
          const int n = top >= lane ? item_span(p, q, rows, top - lane).n : 0;
          int upto = n;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += o;
          }
          const uint32_t hit = __ballot_sync(0xffffffffu, off < upto);
          if (hit) {
            if (lane == __ffs(hit) - 1) {
              ctrl.start_b = b;
              ctrl.start_h = h;
              ctrl.start_tile = top - lane;
              ctrl.start_x = (int)off - (upto - n);
            }
            break;
          }
          off -= __shfl_sync(0xffffffffu, upto, 31);
        }
        break;
      }
    }
    __syncthreads();
  }
  const WaitCtx wc{&ctrl.abort, p.kv.status, p.timeout_ns};
  Place at{};
  at.b = ctrl.start_b;
  if (at.b >= 0) {
    at.h = ctrl.start_h;
    at.tile = ctrl.start_tile;
    at.x = ctrl.start_x;
    at.seq = kv_seq(p.kv, at.b, false);
    at.rows = item_rows(p, at.seq);
    enter_item(p, at);
    at.left = by_item ? at.span.n : (int)(u_end - u_begin);
  }

  if (warp < kSoftmaxWarps) {
    // ================= softmax: a query row per thread =================
    const int tile = warp / kTileWarps;
    const uint32_t lanes = tmem + (uint32_t)(tile * kTileCols) + ((uint32_t)((warp % kTileWarps) * 32) << 16);
    // a row of D fp16 is moved by kLanes lanes of 16 bytes
    constexpr int kLanes = D / 8, kPerRound = 32 / kLanes, kRounds = 32 / kPerRound;
    bool ok = true;
    int stage = 0;          // of the next block of the stripe
    int jt = 0;             // blocks of this tile so far: its places and phases
    int items = 0, cuts = 0;
    long long u = u_begin;  // first block of the piece
    while (ok && at.left > 0) {
    const KvSeq seq = at.seq;
    const int x1 = min(at.span.n, at.x + at.left), pieces = x1 - at.x;  // blocks at.x .. x1 - 1 of the item
    const int first = seq.len - seq.nq, row = at.tile * kRows + warp * 32 + lane;
    const bool live = row < at.rows;
    const int i = live ? kv_div_group(p, row) : 0;
    const int head = at.h * p.group + (live ? row - i * p.group : 0);
    const int pos = first + i;
    const int hi = live ? pos + 1 : 0, lo = p.window > 0 ? pos - p.window + 1 : 0;  // tokens seen
    const Half half_ = tile_half(p, at, tile, at.span.lo + at.x, at.span.lo + x1);

    // Q to shared memory, channels in the codes' order: the warp's 32 rows, kLanes lanes a
    // row (whole lines of global memory); then every row's sum
    const int wrow = (warp % kTileWarps) * 32;  // the warp's first row of the tile
    const long long row_at = live ? (long long)(seq.q0 + i) * p.q_ts + (long long)head * p.q_hs : -1;
    float qsum = 0.f;
    {
      const uint32_t qt = base + Sh::kOffQ + tile * Sh::kQ;
      constexpr int kTogether = 8;  // loads in flight
#pragma unroll 1
      for (int it = 0; it < kRounds; it += kTogether) {
        uint4 v[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const long long from = __shfl_sync(0xffffffffu, row_at, (it + k) * kPerRound + lane / kLanes);
          v[k] = from >= 0 ? *reinterpret_cast<const uint4*>(p.q + from + 8 * (lane % kLanes)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const int r = wrow + (it + k) * kPerRound + lane / kLanes, u = lane % kLanes;
          sts128(qt + (u / 8) * (kTile * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4),
                 make_uint4(__byte_perm(v[k].x, v[k].z, 0x5410), __byte_perm(v[k].y, v[k].w, 0x5410),
                            __byte_perm(v[k].x, v[k].z, 0x7632), __byte_perm(v[k].y, v[k].w, 0x7632)));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ctrl.q_full));
      const int r = wrow + lane;
#pragma unroll
      for (int u = 0; u < kLanes; ++u) {
        const uint4 v = lds128(qt + (u / 8) * (kTile * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4));
        const float2 a = unpack(v.x), bb = unpack(v.y), cc = unpack(v.z), dd = unpack(v.w);
        qsum += ((a.x + a.y) + (bb.x + bb.y)) + ((cc.x + cc.y) + (dd.x + dd.y));
      }
    }
    const F2 qs = dup(qsum);

    float R = live ? kUnset : 0.f;
    F2 l = dup(0.f), pz = dup(0.f);
    const int skipped = half_.to > half_.from ? half_.from - (at.span.lo + at.x) : 0;
    int st = (stage + skipped) % Sh::kStages;
    for (int blk = half_.from; ok && blk < half_.to; ++blk, ++jt) {
      const int t0 = blk * kBlock;
      const uint32_t s_col = lanes + Sh::kColS + (jt & 1) * kBlock;
      if (!wait_warp(bar(ctrl.s_full[tile][jt & 1]), (uint32_t)((jt >> 1) & 1), wc)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* par = reinterpret_cast<const float4*>(par0 + st * (Sh::kPar / 4));
      const bool full = t0 >= half_.all_lo && t0 + kBlock <= half_.all_hi;
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
            const F2 y = mul2(e, {vp.x, vp.y});  // the values' scales and offsets are finite
            pzt = fma2(e, {vp.z, vp.w}, pzt);
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
        const float4 vm = *reinterpret_cast<const float4*>(ctrl.vmax[st]);
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
        if (blk > half_.from && __any_sync(0xffffffffu, f != 1.f)) {
          // once the products of the blocks before are done (this one's follow P)
          if (!wait_warp(bar(ctrl.pv_done[tile]), (uint32_t)((jt - 1) & 1), wc)) break;
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
      if (lane == 0) mbar_arrive(bar(ctrl.p_full[tile][jt & 1]));
      if (++st == Sh::kStages) st = 0;
    }
    // ---- the rows' results, or this CTA's part of them ----
    if (!ok || !wait_warp(bar(ctrl.o_full), (uint32_t)(items & 1), wc)) break;
    tc_fence_after();
    const bool whole = at.x == 0 && x1 == at.span.n;
    const float sum = l.x + l.y, off = pz.x + pz.y;
    const bool any = half_.to > half_.from;  // else there is nothing of this tile in tensor memory
    // a finished row's channels 32 part .. + 31 into Q's room, which no product of this item reads any
    // more.  A warp keeps its 32 rows in the bytes that hold its own rows of Q, as no barrier orders
    // the tile's warps between these rows and the next item's Q: 128 bytes of a row, of 128 channels
    // in two panels, so that rows 0 to 15 of a warp are in the first panel and 16 to 31 in the second.
    // (In the order of Q itself the code of the whole loop came out 5% slower: registers.)
    const uint32_t ot = base + Sh::kOffQ + tile * Sh::kQ - (D == 128 ? wrow * 128 : 0);
    auto place = [&](int r) { return ot + r * (D * 2) + (D == 128 && (r & 16) ? kTile * 128 - 16 * (D * 2) : 0); };
    auto keep = [&](int part, const float (&v)[32]) {
      const int r = wrow + lane;
#pragma unroll
      for (int t = 0; t < 32; t += 8) {
        const int u = part * 4 + t / 8;
        sts128(place(r) + ((u ^ (r & 7)) << 4), make_uint4(pack(v[t], v[t + 1]), pack(v[t + 2], v[t + 3]),
                                                                   pack(v[t + 4], v[t + 5]), pack(v[t + 6], v[t + 7])));
      }
    };
    // the warp's rows from there to the output, whole lines at a time
    const long long out_at = live ? ((long long)(seq.q0 + i) * p.heads + head) * D : -1;
    auto write_rows = [&]() {
      __syncwarp();
#pragma unroll 4
      for (int it = 0; it < kRounds; ++it) {
        const int r = it * kPerRound + lane / kLanes, u = lane % kLanes;
        const long long to = __shfl_sync(0xffffffffu, out_at, r);
        const uint4 v = lds128(place(wrow + r) + ((u ^ (r & 7)) << 4));
        if (to >= 0) *reinterpret_cast<uint4*>(p.out + to + 8 * u) = v;
      }
      __syncwarp();
    };
    if (whole) {
      const float inv = hi > 0 ? 1.f / sum : 0.f, add = off * inv;  // a row that sees no token is zero
#pragma unroll 1
      for (int part = 0; part < D / 32; ++part) {
        uint32_t v[32];
        tmem_ld32(lanes + Sh::kColO + part * 32, v);
        tmem_wait_ld();
        float o[32];
#pragma unroll
        for (int t = 0; t < 32; ++t) o[t] = fmaf(__uint_as_float(v[t]), inv, add);
        if (inv == 0.f) {  // also where tensor memory holds nothing of this tile
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = 0.f;
        }
        keep(part, o);
      }
      write_rows();
    } else {
      // slot 0: a piece of an item that began before this stripe; slot 1: the beginning of one.
      // Channel-major, so that a warp's rows are written and read in whole lines.
      constexpr int kSlot = kRows * (D + 4);
      const int my_row = warp * 32 + lane;
      float* slot = p.partials + (2ll * blockIdx.x + (at.x == 0 ? 1 : 0)) * kSlot + my_row;
#pragma unroll 1
      for (int part = 0; part < D / 32; ++part) {
        uint32_t v[32];
        tmem_ld32(lanes + Sh::kColO + part * 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int t = 0; t < 32; ++t) __stcg(slot + (part * 32 + t) * kRows, any ? __uint_as_float(v[t]) + off : 0.f);
      }
      __stcg(slot + D * kRows, R);
      __stcg(slot + (D + 1) * kRows, sum);
      // all warps have written; one thread counts this CTA in, with release and acquire for all of them
      const long long s0 = u - at.x;  // the item's first block among all
      const int c0 = (int)stripe_owner(s0, U, G), c1 = (int)stripe_owner(s0 + at.span.n - 1, U, G);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(ctrl.part_done));
      if (warp == 0) {
        if (!wait_warp(bar(ctrl.part_done), (uint32_t)(cuts & 1), wc)) break;
        if (lane == 0) {
          int arrived;
          asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                       : "=r"(arrived)
                       : "l"(p.counters + c0)
                       : "memory");
          ctrl.last = arrived == c1 - c0;
          if (ctrl.last) p.counters[c0] = 0;  // all are here: ready for the next call
          mbar_arrive(bar(ctrl.verdict));
        }
        __syncwarp();
      }
      if (!wait_warp(bar(ctrl.verdict), (uint32_t)(cuts & 1), wc)) break;
      ++cuts;
      if (*reinterpret_cast<volatile int*>(&ctrl.last)) {
        // the parts in stripe order: the first CTA's is its slot 1, the others' their slot 0
        auto part_of = [&](int q) { return p.partials + (2ll * q + (q == c0 ? 1 : 0)) * kSlot + my_row; };
        float top = kUnset, all = 0.f;
        for (int q = c0; q <= c1; ++q) {
          const float r = __ldcg(part_of(q) + D * kRows), lq = __ldcg(part_of(q) + (D + 1) * kRows);
          const float nt = lq == 0.f ? top : fmaxf(top, r);
          all = fmaf(all, top == nt ? 1.f : ex2(top - nt), lq == 0.f ? 0.f : r == nt ? lq : lq * ex2(r - nt));
          top = nt;
        }
        const float inv = hi > 0 ? 1.f / all : 0.f;
#pragma unroll 1
        for (int part = 0; part < D / 32; ++part) {
          float o[32];
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = 0.f;
#pragma unroll 1
          for (int q = c0; q <= c1; ++q) {
            const float r = __ldcg(part_of(q) + D * kRows), lq = __ldcg(part_of(q) + (D + 1) * kRows);
            const float f = lq == 0.f ? 0.f : r == top ? 1.f : ex2(r - top);
#pragma unroll
            for (int t = 0; t < 32; ++t) o[t] = fmaf(__ldcg(part_of(q) + (part * 32 + t) * kRows), f, o[t]);
          }
#pragma unroll
          for (int t = 0; t < 32; ++t) o[t] = inv == 0.f ? 0.f : o[t] * inv;
          keep(part, o);
        }
        write_rows();
      }
    }
    // on to the next item; its Q may replace this one's: o_full followed all products
    tc_fence_before();
    ++items;
    stage = (stage + pieces) % Sh::kStages;
    u += pieces;
    move_on(p, at, pieces);
    }
  } else if (warp < kSoftmaxWarps + kDequantWarps) {
    // ================= dequantisation =================
    const int dw = warp - kSoftmaxWarps, g = lane >> 2, c = lane & 3;
    const int half = dw >> 1, wp = dw & 1;  // this warp's part of the values
    // warp 0 of the four keeps kRing blocks in flight: lane q < 4 copies granule q
    const uint64_t policy = policy_evict_last();  // other CTAs read the same blocks
    const uint32_t raw = base + Sh::kOffRaw;
    const int n = at.left;
    Place ahead = at;  // the next block to copy
    int next_page = 0, issued = 0;
    auto look_up = [&]() {
      const int gi = (ahead.span.lo + ahead.x) * 4 + lane;
      if (lane < 4 && gi * kGranule < ahead.seq.len)
        next_page = p.kv.table[(long long)ahead.b * p.kv.max_pages + kv_div_page(p.kv, gi)];
    };
    auto issue = [&]() {
      const int gi = (ahead.span.lo + ahead.x) * 4 + lane, slot = issued % Sh::kRing;
      const bool inside = lane < 4 && gi * kGranule < ahead.seq.len;
      const bool there = inside && (uint32_t)next_page < (uint32_t)p.kv.n_pages;
      if (inside && !there) kv_fail(p.kv, kKvSitePage);  // no copy: the results are not valid, and reported
      const int copies = __popc(__ballot_sync(0xffffffffu, there));
      if (lane == 0) mbar_arrive_expect_tx(bar(ctrl.raw_full[slot]), copies * GR);
      __syncwarp();
      if (there && (lane == 0 || !p.whole_blocks))
        bulk_g2s(raw + slot * Sh::kRaw + lane * GR,
                 p.kv.cache + ahead.h * p.kv.head_bytes + next_page * p.kv.page_bytes +
                     (gi - kv_div_page(p.kv, gi) * p.kv.page16) * GR,
                 p.whole_blocks ? copies * GR : GR, bar(ctrl.raw_full[slot]), policy);
      if (++issued < n) {
        move_on(p, ahead, 1);
        look_up();
      }
    };
    if (dw == 0 && n > 0) {
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
      if (lane < 16 && ((at.span.lo + at.x) * 4 + dw) * kGranule + lane < at.seq.len)
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
        float2 kf = unpack(pr.x), vf = unpack(pr.y);
        if (!(fabsf(vf.x) <= 65504.f)) {  // a value that holds NaN: by way of its score, which masks can take out
          kf.x = vf.x;
          vf.x = vf.y = 0.f;
        }
        float big = lane < 16 ? vf.x : 0.f;
        #pragma unroll
        for (int m = 1; m < 16; m <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
        if (lane < 16) {
          float* dst = par0 + stage * (Sh::kPar / 4) + (16 * dw + (lane & ~1)) * 4 + (lane & 1);
          dst[0] = kf.x * p.scale_log2;
          dst[2] = kf.y * p.scale_log2;
          // no less than 2^-30, so that p s shows how far a row's reference is behind: a vector of
          // scale 0 has codes less 8 of 0, whose product with any p s is none, and no other
          // scale is below fp16's 2^-24
          dst[4] = fmaxf(vf.x, kLeastScale);
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
      move_on(p, at, 1);
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
    int stage = 0;           // of block blk
    uint32_t ph = 0;
    int jt[kTiles] = {0, 0};  // blocks of each tile whose products with V were issued: places and phases
    int items = 0;
    bool ok = true;
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
    while (ok && at.left > 0) {
      const int pieces = min(at.span.n - at.x, at.left), blk0 = at.span.lo + at.x, end = blk0 + pieces;
      Half half_[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) half_[t] = tile_half(p, at, t, blk0, end);
      // Q of this item, which the softmax warps write after the item before is done
      if (!(ok = wait_warp(bar(ctrl.q_full), (uint32_t)(items & 1), wc))) break;
      if (!(ok = wait_warp(bar(ctrl.kv_full[stage]), ph, wc))) break;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (half_[t].from == blk0 && half_[t].to > blk0) scores(t, jt[t], stage);
      for (int blk = blk0; ok && blk < end; ++blk) {
        int next = stage + 1;
        uint32_t next_ph = ph;
        if (next == Sh::kStages) {
          next = 0;
          next_ph ^= 1u;
        }
        if (blk + 1 < end) {  // the next block's scores go before this one's products with V
          if (!(ok = wait_warp(bar(ctrl.kv_full[next]), next_ph, wc))) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
            if (blk + 1 >= half_[t].from && blk + 1 < half_[t].to) scores(t, jt[t] + (blk >= half_[t].from), next);
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          if (!ok || blk < half_[t].from || blk >= half_[t].to) continue;
          const int i = jt[t];
          if (!(ok = wait_warp(bar(ctrl.p_full[t][i & 1]), (uint32_t)((i >> 1) & 1), wc))) continue;
          tc_fence_after();
          const uint32_t cols = tmem + t * kTileCols;
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            mma_f16_ts_elect(cols + Sh::kColO, cols + Sh::kColS + (i & 1) * kBlock + kk * 8,
                             umma_desc_sw128(base + Sh::kOffV + stage * Sh::kV) + (uint64_t)(2 * kk), id_o,
                             blk > half_[t].from || kk > 0);
          mma_commit_elect(bar(ctrl.pv_done[t]));
          ++jt[t];
        }
        if (!ok) break;
        mma_commit_elect(bar(ctrl.kv_empty[stage]));
        stage = next;
        ph = next_ph;
      }
      if (!ok) break;
      mma_commit_elect(bar(ctrl.o_full));
      ++items;
      move_on(p, at, pieces);
    }
    mma_commit_elect(bar(ctrl.drain));
    wait_drain(bar(ctrl.drain), 0, wc);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftmaxWarps + kDequantWarps) tmem_dealloc(tmem, kTmem);
}

template <int D>
cudaError_t launch(const KvAttnParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
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

cudaError_t launch_kv_prefill(const KvAttnParams& p, int D, int grid, cudaStream_t stream) {
  return D == 128 ? launch<128>(p, grid, stream) : launch<64>(p, grid, stream);
}

}  // namespace w4a16
