// kv_attn.cu -- causal attention of new tokens over the 4-bit paged cache, for
// few query rows per key head (single tokens, a few proposed ones):
//     O[i][h] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q[i][h] . k_t - max),
// over the cached tokens t <= position(i) (and t > position(i) - window).
//
// Bound: streaming the cache, 2 (D/2 + 4) bytes per token and key head, once.
//   * The work is (request, key head, group of 8 NB query rows) segments of
//     blocks of 64 tokens; the rows of a group are the query heads that share
//     the key head, for one or more query tokens, so that a block is read once
//     for all of them.  Every warp of the card takes an equal contiguous stripe
//     of blocks, found on the device from the lengths, with its own ring of
//     bulk copies, running maximum, sum and accumulators: no barrier until the
//     stripe is done.
//   * Both products run on mma.sync with the cache as the 16-row operand and the
//     query rows as the 8 columns: S^T[16 tokens x 8 rows] = K Q^T and
//     O^T[16 channels x 8 rows] += V^T P^T.  A code c is fed as the fp16
//     subnormal c * 2^-24 (one AND per pair; the nibble four bits up is
//     16 c * 2^-24): the products are exact and scales, offsets and the powers
//     of two are applied to the fp32 results (kv.cuh has the algebra).
//   * p_t s_t is fed as the sum of two fp16 numbers (22 bits): the result is then
//     as near to 64 bits as its own rounding leaves it (2.1e-4 of it in root mean
//     square, 2.3e-4 at 131,001 tokens), where one fp16 number, as in the prompt
//     kernel, gives 2.7 to 3.0e-4.  s_t is normalised by a running power of two so
//     that neither half falls below fp16's range.
//   * The maximum is only moved when a score exceeds it by 2^8 (one vote per
//     block instead of shuffles and a rescaling).
// A segment that is one warp's alone is written by that warp; the parts of one
// that is cut between warps meet in shared memory; one that is cut between CTAs
// is finished by whichever of them arrives last, summing all parts in stripe
// order (so the result does not depend on the order of arrival).  Nothing waits
// for another CTA.
//
// Measured: 40 requests of up to 7900 tokens, 64 query heads on 8 of 128 channels,
// 55.8 us, 222 MB, 4.0 TB/s (60% of the card's copy rate); one request of 131,001
// tokens 39 us, 143 MB, 3.6 TB/s; one of 700 tokens, 32 heads (32 segments of 11
// blocks, a CTA each), 10.5 us, which is latency: the look-ups and the first copy, a
// block or two a warp, the join of its eight warps.  40 requests with 16 query rows a
// key head (two row groups an instruction): 98 us under ncu, where 8 rows take 61.
// The stream alone, without the arithmetic, takes
// 28 us of the first case; the arithmetic, 122 instructions of two cycles and 26 mma of
// eight for a granule and warp, takes most of the rest.  Blocks of 64 tokens,
// eight warps, rings of two blocks (four at 64 channels): more warps, longer rings
// and smaller blocks measured the same or up to 10% slower.
#include <type_traits>

#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLowest = -1e30f;       // the running maximum before the first score
constexpr float kLazy = 8.f;            // log2 of how far a score may exceed the reference
constexpr float kCodeUnit = 16777216.f;  // 2^24: an fp16 subnormal's unit is 2^-24
constexpr uint32_t kEight = 0x80088008u;  // a pair of -8 of these units
constexpr float kMinSref = 9.313225746154785e-10f;  // 2^-30

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// Plain loads from shared memory (the compiler may move them up to the wait).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(at);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(at);
    w[0] = v.x; w[1] = v.y;
  }
}

// Four channels of an output row: row rr of key head h, normalised.  A row
// that sees no token is zero; of trees' rows kv_tree_sum tells by their sum.
template <bool kTree>
__device__ __forceinline__ void store_row(const KvAttnParams& p, const KvSeq& s, int h, int rr, int ch, int D,
                                          float4 acc, float sum) {
  const int i = kv_div_group(p, rr), head = h * p.group + rr - i * p.group;
  const float inv = kTree || s.len - s.nq + i >= 0 ? 1.f / sum : 0.f;
  if (inv == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
  uint2 v;
  v.x = h2_bits(__floats2half2_rn(acc.x * inv, acc.y * inv));
  v.y = h2_bits(__floats2half2_rn(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(p.out + ((long long)(s.q0 + i) * p.heads + head) * D + ch) = v;
}

// Pairs of fp32 values: one instruction for two operations, where both
// operands are pairs already (at two cycles it costs the pipe what two scalar
// operations do, and duplicating an operand would cost moves on the busier one).
struct F2 {
  float x, y;
};
__device__ __forceinline__ void mma16816(F2 (&d)[2], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0].x), "+f"(d[0].y), "+f"(d[1].x), "+f"(d[1].y)
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

// W warps; blocks of GB granules, GI of them taken together; S blocks in a warp's ring.
// kT: the new tokens are trees: blocks that hold some of them, or where a window begins, take their masks from the
// rows' bits (kv.cuh).  Measured: a tree of 8 on 692 tokens, 32 heads of 128 channels, 10.9 us; 24 of 5, window
// 2048, 24 heads on 8 of 64 channels, 26.8 us.
template <int D, int NB, bool kT>
struct Shape {
  static constexpr bool kTree = kT;
  static constexpr int W = 8, GB = 4, GI = NB == 1 ? 4 : 2, S = D == 128 ? 2 : 4;
  static constexpr int kBlock = GB * kGranule;  // tokens
  static constexpr int kStep = GI * kGranule;  // tokens taken together
  static constexpr int RB = 8 * NB;             // query rows
  static constexpr int GR = kv_granule_bytes(D);
  static constexpr int BB = GB * GR;            // bytes of a block
  static constexpr int kOStride = D + 4;        // floats of a row of a part in shared memory
  static constexpr int kPart = RB * (kOStride + 2) * 4;  // rows, then (maximum, sum) of each
  // Units that a segment's start counts for beside its blocks where the work is cut into equal shares: the queries,
  // the masks where a window begins and new tokens are, the parts.  Of trees alone: measured with 15 rows a key head
  // of 64 channels, window 2048, 20 requests 23.7 us, 26.5 without, 24 26.6 / 28.8, 38 34.6 / 36.0, 100 70.1 / 70.1;
  // 20 trees of 8 on 692 tokens, 32 heads of 128 channels, 26.8 / 29.3; 24 of 5 on 500 16.0 / 15.6 (finding the shares).
  static constexpr int kStart = kTree ? 3 : 0;
  static constexpr int kRing = 3 * 1024;          // after the control block
  static constexpr int kSmem = kRing + W * S * BB;
  static_assert(kPart <= S * BB && kPart % 16 == 0, "a part has to fit a warp's ring");
  static_assert(W <= kKvAttnWarps && W * S <= 64, "the control block's and the workspace's room");
};

// One request's share of the work: its blocks [lo, lo + n) and the number of
// its groups of query rows.
struct SeqWork {
  KvSeq s;
  int lo, n, rbs;
};

template <typename Sh>
__device__ __forceinline__ SeqWork seq_work(const KvAttnParams& p, int b, bool report) {
  SeqWork w;
  w.s = kv_seq(p.kv, b, report);
  if (w.s.nq > w.s.len && report) kv_fail(p.kv, kKvSiteLen);
  if (Sh::kTree && report && w.s.nq > 32ll * p.tree_words) kv_fail(p.kv, kKvSiteTree);
  const int rows = w.s.nq * p.group;
  w.rbs = rows > p.max_rows ? 0 : (rows + Sh::RB - 1) / Sh::RB;
  const int first = w.s.len - w.s.nq;  // position of the first query token
  // (a row of a tree that saw no new token would be at first - 1)
  const int lo = p.window > 0 ? max(0, first - p.window + (Sh::kTree ? 0 : 1)) : 0;
  w.lo = lo / Sh::kBlock;
  w.n = max(1, (w.s.len + Sh::kBlock - 1) / Sh::kBlock - w.lo);
  return w;
}

// A place in the stripe: block g of segment seg (key head * rbs + row group) of
// request b.
struct Cursor {
  int b, seg, g;
  SeqWork w;
};

template <typename Sh, int kStart = 0>
__device__ __forceinline__ void advance(const KvAttnParams& p, Cursor& c, int by) {
  c.g += by;
  while (c.g >= c.w.n + kStart) {
    c.g -= c.w.n + kStart;
    if (++c.seg == p.kv.hkv * c.w.rbs) {
      c.seg = 0;
      do {
        if (++c.b >= p.kv.B) { c.g = 0; return; }
        c.w = seq_work<Sh>(p, c.b, false);
      } while (c.w.rbs == 0);
    }
  }
}

// Moves on by k segments, to the beginning of one.
template <typename Sh>
__device__ __forceinline__ void skip_segments(const KvAttnParams& p, Cursor& c, int k) {
  c.g = 0;
  c.seg += k;
  while (c.seg >= p.kv.hkv * c.w.rbs) {
    c.seg -= p.kv.hkv * c.w.rbs;
    do {
      if (++c.b >= p.kv.B) return;
      c.w = seq_work<Sh>(p, c.b, false);
    } while (c.w.rbs == 0);
  }
}

// What a warp left in shared memory: the end of a segment that began before its
// stripe (or a middle of one), and the beginning of one that goes on after it.
struct Segment {
  KvSeq s;                 // its request's rows and length
  int h, rb, n;            // key head, group of query rows, blocks
  long long s0;            // first unit
};
struct Parts {
  int idle;                // the warp has no blocks
  int first, last;         // whether there is one
  int first_ends;          // the segment ends in this warp
  int first_last;          // nothing comes after it in the stripe: it is in the ring, else in the workspace
  Segment seg[2];          // of first and last
};

// Joins one part's (maximum, sum) and values of four channels.  A part that saw
// no token has sum 0 and zeros.
__device__ __forceinline__ void join(float2 ml, float4 a, float& top, float& sum, float4& acc) {
  const float nt = ml.y == 0.f ? top : fmaxf(top, ml.x);
  const float fo = top == nt ? 1.f : ex2(top - nt), fn = ml.x == nt ? 1.f : ml.y == 0.f ? 0.f : ex2(ml.x - nt);
  top = nt;
  sum = fmaf(sum, fo, ml.y * fn);
  acc.x = fmaf(acc.x, fo, a.x * fn);
  acc.y = fmaf(acc.y, fo, a.y * fn);
  acc.z = fmaf(acc.z, fo, a.z * fn);
  acc.w = fmaf(acc.w, fo, a.w * fn);
}

// stripe_begin and stripe_owner, in 32 bits where the products fit.
__device__ __forceinline__ long long begin_of(long long i, long long U, long long N) {
  return U * N < (1ll << 32) ? (long long)((uint32_t)(i * U) / (uint32_t)N) : stripe_begin(i, U, N);
}
__device__ __forceinline__ long long owner_of(long long u, long long U, long long N) {
  return U * N < (1ll << 32) ? (long long)((uint32_t)((u + 1) * N - 1) / (uint32_t)U) : stripe_owner(u, U, N);
}

struct AttnCtrl {
  uint64_t full[64];       // [W][S]
  long long scan[16], scan_segs[16];
  int longest[16];
  long long start_off;     // the first unit's offset in its request
  int start_b;
  int abort;
  int arrived[2];
  SeqWork start_w;
  Parts parts[kKvAttnWarps];
};
static_assert(sizeof(AttnCtrl) <= 3 * 1024, "control block too large");

template <int D, int NB, bool kTree>
__global__ void __launch_bounds__(Shape<D, NB, kTree>::W * 32, 1) kv_attn_kernel(const KvAttnParams p) {
  using Sh = Shape<D, NB, kTree>;
  constexpr int W = Sh::W, S = Sh::S, GB = Sh::GB, GI = Sh::GI, RB = Sh::RB, GR = Sh::GR, BB = Sh::BB, CW = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  AttnCtrl* ctrl = reinterpret_cast<AttnCtrl*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* const ring_ptr = smem + Sh::kRing + warp * (S * BB);
  const uint32_t ring = smem_addr(ring_ptr);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(smem_addr(&ctrl->full[warp * S + s]), 1);
    ctrl->parts[warp].first = ctrl->parts[warp].last = 0;
    if (warp == 0) ctrl->abort = 0;
    fence_mbarrier_init();
  }
  if (tid == 0) griddep_launch_dependents();
  kv_prefetch_plan(p.kv, (long long)blockIdx.x * (W * 32) + tid);
  griddep_wait();

  // ---- the stripes: all blocks, and this CTA's and this warp's -----------------
  const int per = (p.kv.B + W * 32 - 1) / (W * 32);
  const int b0 = min(tid * per, p.kv.B), b1 = min(b0 + per, p.kv.B);
  long long mine = 0, mine_segs = 0;
  int longest = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqWork w = seq_work<Sh>(p, b, blockIdx.x == 0);
    const long long segs = (long long)p.kv.hkv * w.rbs;
    mine += segs * (w.n + Sh::kStart);
    mine_segs += segs;
    if (segs) longest = max(longest, w.n);
  }
  long long before = mine, before_segs = mine_segs;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, before, m), os = __shfl_up_sync(0xffffffffu, before_segs, m);
    if (lane >= m) {
      before += o;
      before_segs += os;
    }
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, m));
  }
  if (lane == 31) {
    ctrl->scan[warp] = before;
    ctrl->scan_segs[warp] = before_segs;
    ctrl->longest[warp] = longest;
  }
  __syncthreads();
  long long U = 0, segs = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == warp) {
      before += U - mine;
      before_segs += segs - mine_segs;
    }
    U += ctrl->scan[w];
    segs += ctrl->scan_segs[w];
    longest = max(longest, ctrl->longest[w]);
  }
  if (U == 0) return;
  // Few short segments: a CTA each (by_seg), so that none is cut between CTAs.  Many: a
  // run of whole ones for every warp (by_warp), so that none is cut at all.  What that
  // may cost a warp in blocks is what publishing and joining parts costs: 2 between CTAs,
  // 4 with those between warps, half of it where a block is of 16 rows.  Measured with
  // 128 channels, whole against cut: 32 segments of 32 blocks (4 a warp, cut 1) 14.4
  // against 12.2 us, 64 of 65 (9, 3) 23.4 against 18.7; 256 of 4 blocks (4, 1) 13.7
  // against 14.9, 1536 of 2 (4, 3) 16.4 against 23.5.
  constexpr int kCutSeg = NB == 1 ? 2 : 1, kCutWarp = NB == 1 ? 4 : 2;
  const long long warps = (long long)gridDim.x * W, even = (U - segs * Sh::kStart + warps - 1) / warps;
  const bool by_seg = segs <= (long long)gridDim.x && (longest + W - 1) / W <= even + kCutSeg;
  const bool by_warp = segs > (long long)gridDim.x && (segs + warps - 1) / warps * longest <= even + kCutWarp;
  const bool uncut = by_seg || by_warp;
  // otherwise an equal share of all units for every warp, at least one
  const long long G = by_seg ? segs : by_warp ? gridDim.x : min((long long)gridDim.x, (U + W - 1) / W);
  if (blockIdx.x >= G) return;
  const long long u_cta = begin_of(blockIdx.x, U, G);
  {
    const long long at = by_seg ? blockIdx.x : by_warp ? begin_of(blockIdx.x, segs, G) : u_cta;
    const long long from = uncut ? before_segs : before;
    if (at >= from && at < from + (uncut ? mine_segs : mine)) {
      long long off = at - from;
      for (int b = b0; b < b1; ++b) {
        const SeqWork w = seq_work<Sh>(p, b, false);
        const long long n = (long long)p.kv.hkv * w.rbs * (uncut ? 1 : w.n + Sh::kStart);
        if (off < n) {
          ctrl->start_b = b;
          ctrl->start_w = w;
          ctrl->start_off = uncut ? off * w.n : off;
          break;
        }
        off -= n;
      }
    }
  }
  __syncthreads();
  Cursor cur;
  cur.b = ctrl->start_b;
  cur.w = ctrl->start_w;
  const long long start_off = ctrl->start_off;
  const int weight = cur.w.n + (uncut ? 0 : Sh::kStart);
  cur.seg = start_off < (1ll << 32) ? (int)((uint32_t)start_off / (uint32_t)weight) : (int)(start_off / weight);
  cur.g = (int)(start_off - (long long)cur.seg * weight);
  int total;           // this warp's blocks
  long long from = 0;  // and the first of them; of trees' equal shares: the first unit of its first segment
  if (by_seg) {
    from = (long long)cur.w.n * warp / W;
    total = (int)((long long)cur.w.n * (warp + 1) / W - from);
    cur.g += (int)from;  // inside the segment, or at its end where there is nothing left to do
  } else if (by_warp) {
    const long long gw = (long long)blockIdx.x * W + warp, s0 = begin_of(gw, segs, G * W);
    int left = (int)(begin_of(gw + 1, segs, G * W) - s0);
    total = 0;
    if (left > 0) {
      skip_segments<Sh>(p, cur, (int)(s0 - begin_of(blockIdx.x, segs, G)));
      for (Cursor c = cur; left > 0;) {
        const int take = min(left, p.kv.hkv * c.w.rbs - c.seg);
        total += take * c.w.n;
        left -= take;
        if (left > 0) skip_segments<Sh>(p, c, take);
      }
    }
  } else {
    const long long gw = (long long)blockIdx.x * W + warp;
    from = begin_of(gw, U, G * W);
    total = (int)(begin_of(gw + 1, U, G * W) - from);
    if (total > 0) advance<Sh, Sh::kStart>(p, cur, (int)(from - u_cta));
    if constexpr (Sh::kStart > 0) {  // from units to blocks
      int left = total;
      total = 0;
      for (Cursor c = cur; left > 0;) {
        const int take = min(left, c.w.n + Sh::kStart - c.g);
        total += max(c.g + take - max(c.g, Sh::kStart), 0);
        left -= take;
        if (left > 0) advance<Sh, Sh::kStart>(p, c, take);
      }
      from -= cur.g;  // the segment's first unit
      cur.g = max(cur.g - Sh::kStart, 0);
    }
  }

  if (lane == 0) ctrl->parts[warp].idle = total == 0;
  const uint64_t policy = policy_evict_first();  // the cache is read once
  const WaitCtx wc{&ctrl->abort, p.kv.status, p.timeout_ns};

  // ---- the ring's producer: lane i < GB copies granule i of the next block -------------
  Cursor pc = cur;
  const int* table = nullptr;  // the request's pages
  uint8_t* heads = nullptr;    // the key head's place in page 0
  int gi = 0, issued = 0, next_page = 0;  // this lane's granule, blocks copied, the granule's page
  auto enter = [&]() {  // a new segment
    table = p.kv.table + (long long)pc.b * p.kv.max_pages;
    heads = p.kv.cache + (pc.seg / pc.w.rbs) * p.kv.head_bytes;
    gi = (pc.w.lo + pc.g) * GB + lane;
  };
  auto look_up = [&]() {
    if (lane < GB && gi * kGranule < pc.w.s.len) next_page = table[kv_div_page(p.kv, gi)];
  };
  auto issue = [&](int stage) {
    const bool inside = lane < GB && gi * kGranule < pc.w.s.len;
    const bool there = inside && (uint32_t)next_page < (uint32_t)p.kv.n_pages;
    if (inside && !there) kv_fail(p.kv, kKvSitePage);  // no copy: the block's results are not valid, and reported
    const int n = __popc(__ballot_sync(0xffffffffu, there));
    const uint32_t bar = smem_addr(&ctrl->full[warp * S + stage]);
    if (lane == 0) mbar_arrive_expect_tx(bar, n * GR);
    __syncwarp();
    if (there && (lane == 0 || !p.whole_blocks))
      bulk_g2s(ring + stage * BB + lane * GR,
               heads + next_page * p.kv.page_bytes + (gi - kv_div_page(p.kv, gi) * p.kv.page16) * GR,
               p.whole_blocks ? n * GR : GR, bar, policy);
    if (++issued < total) {
      gi += GB;
      if (++pc.g == pc.w.n) {
        pc.g -= 1;
        advance<Sh>(p, pc, 1);
        enter();
      }
      look_up();
    }
  };
  if (total > 0) {
    enter();
    look_up();
  }
  while (issued < min(S, total)) issue(issued);

  int done = 0;  // blocks of this warp consumed
  bool ok = true;
  while (ok && done < total) {
    const SeqWork& w = cur.w;
    const int cnt = min(total - done, w.n - cur.g);
    const int h = cur.seg / w.rbs, rb = cur.seg - h * w.rbs;
    const int rows = w.s.nq * p.group;
    const int first = w.s.len - w.s.nq;

    // ---- queries: B operands in the channel order of the codes, and their sums ----
    uint32_t qf[NB][CW * 4];
    F2 qs[NB];
    int hi_pos[NB][2], lo_pos[NB][2];  // tokens seen by rows 2c, 2c + 1: [lo, hi); of trees: hi is the row's new token
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = rb * RB + nb * 8 + g;
      float sum = 0.f;
      if (row < rows) {
        const int i = kv_div_group(p, row), head = h * p.group + row - i * p.group;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + (long long)(w.s.q0 + i) * p.q_ts + (long long)head * p.q_hs + c * (D / 4));
#pragma unroll
        for (int j = 0; j < CW; ++j) {
          const uint4 v = src[j];  // channels 8j .. 8j + 7 of the lane's
          qf[nb][4 * j + 0] = __byte_perm(v.x, v.z, 0x5410);  // 0, 4
          qf[nb][4 * j + 1] = __byte_perm(v.y, v.w, 0x5410);  // 2, 6
          qf[nb][4 * j + 2] = __byte_perm(v.x, v.z, 0x7632);  // 1, 5
          qf[nb][4 * j + 3] = __byte_perm(v.y, v.w, 0x7632);  // 3, 7
          const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[k]));
            sum += f.x + f.y;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < CW * 4; ++j) qf[nb][j] = 0u;
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qs[nb].x = __shfl_sync(0xffffffffu, sum, 8 * c) * p.scale_log2;
      qs[nb].y = __shfl_sync(0xffffffffu, sum, 8 * c + 4) * p.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = rb * RB + nb * 8 + 2 * c + e;
        if constexpr (kTree) {
          hi_pos[nb][e] = rr < rows ? kv_div_group(p, rr) : -1;
          lo_pos[nb][e] = rr < rows ? kv_tree_lo(p, w.s, hi_pos[nb][e]) : 0;
        } else {
          const int pos = first + kv_div_group(p, rr);
          hi_pos[nb][e] = rr < rows ? pos + 1 : 0;
          lo_pos[nb][e] = p.window > 0 ? pos - p.window + 1 : 0;
        }
      }
    }
    // tokens every row sees, [all_lo, all_hi), and tokens any row sees
    const int i_first = kv_div_group(p, rb * RB), i_last = kv_div_group(p, min(rows, (rb + 1) * RB) - 1);
    const int all_hi = kTree ? first : first + i_first + 1, any_hi = kTree ? w.s.len : first + i_last + 1;
    const int all_lo = p.window > 0 ? first + (kTree ? w.s.nq - 1 : i_last) - p.window + 1 : 0;
    const int any_lo = p.window > 0 ? first + (kTree ? -1 : i_first) - p.window + 1 : 0;

    F2 m[NB], l[NB], pz[NB], o[CW * 2][NB][2];  // o: rows g and g + 8 of the tile
    float sref = kMinSref;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      m[nb] = dup(kLowest);
      l[nb] = pz[nb] = dup(0.f);
#pragma unroll
      for (int t = 0; t < CW * 2; ++t) o[t][nb][0] = o[t][nb][1] = dup(0.f);
    }

    auto block = [&](auto masked, const int t0, const uint8_t* st) {
      using Masked = decltype(masked);

      // trees: which tokens rows 2c, 2c + 1 see; bit 16 (q & 1) + 8 e of word q / 2 is this lane's token g + 8 e of granule q
      // of `any`: whether some row of the warp's sees it
      uint32_t see[NB][2][Sh::kStep / 32], any[Sh::kStep / 32];
      if constexpr (kTree && Masked::value) {
#pragma unroll
        for (int k = 0; k < Sh::kStep / 32; ++k) {
          any[k] = 0u;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t all = hi_pos[nb][r] >= 0 ? kv_tree_see(p, w.s, hi_pos[nb][r], lo_pos[nb][r], t0 + 32 * k) : 0u;
              any[k] |= all;
              see[nb][r][k] = all >> g;
            }
          any[k] |= __shfl_xor_sync(0xffffffffu, any[k], 1);
          any[k] |= __shfl_xor_sync(0xffffffffu, any[k], 2);
          any[k] >>= g;
        }
      }
      auto hidden = [&](int nb, int r, int q, int e) {
        if constexpr (kTree && Masked::value) return !((see[nb][r][q / 2] >> (16 * (q & 1) + 8 * e)) & 1u);
        const int t = t0 + 16 * q + g + 8 * e;
        return t >= hi_pos[nb][r] || t < lo_pos[nb][r];
      };

      // ---- S^T = K Q^T on the codes: low nibbles and high (x 16) apart -----------
      // x: scores in units of log2; element (q, nb, e) is token g + 8 e of granule
      // q for rows 2c, 2c + 1
      F2 x[GI][NB][2], top[NB];
      float vs[GI][2], vo[GI][2], big = 0.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) top[nb] = dup(kLowest);
      uint32_t k0[GI][CW], k1[GI][CW];
      F2 sl[GI][NB][2], sh[GI][NB][2];
#pragma unroll
      for (int q = 0; q < GI; ++q) {
        load_words<CW>(st + q * GR + g * (D / 2) + c * (D / 8), k0[q]);
        load_words<CW>(st + q * GR + (g + 8) * (D / 2) + c * (D / 8), k1[q]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) sl[q][nb][0] = sl[q][nb][1] = sh[q][nb][0] = sh[q][nb][1] = dup(0.f);
      }
      // the granules in turn, so that no product waits for the one before
#pragma unroll
      for (int j = 0; j < CW; ++j)
#pragma unroll
        for (int q = 0; q < GI; ++q) {
          const uint32_t a0 = k0[q][j], a1 = k1[q][j], a2 = k0[q][j] >> 8, a3 = k1[q][j] >> 8;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma16816(sl[q][nb], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a2 & 0x000F000Fu, a3 & 0x000F000Fu,
                     qf[nb][4 * j], qf[nb][4 * j + 1]);
            mma16816(sh[q][nb], a0 & 0x00F000F0u, a1 & 0x00F000F0u, a2 & 0x00F000F0u, a3 & 0x00F000F0u,
                     qf[nb][4 * j + 2], qf[nb][4 * j + 3]);
          }
        }
#pragma unroll
      for (int q = 0; q < GI; ++q) {
        uint32_t pr[2][2];
        load_words<2>(st + q * GR + 16 * D + g * 8, pr[0]);
        load_words<2>(st + q * GR + 16 * D + (g + 8) * 8, pr[1]);
        // scales and offsets of tokens g and g + 8; nothing is taken from slots
        // that no row sees (they may hold anything)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&pr[e][0]));
          const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&pr[e][1]));
          float ks = kf.x * (kCodeUnit * p.scale_log2), kz = fmaf(-8.f, kf.x, kf.y);
          vs[q][e] = vf.x;
          vo[q][e] = vf.y;
          const int t = t0 + 16 * q + g + 8 * e;
          bool unseen = Masked::value && (t >= any_hi || t < any_lo);
          if constexpr (kTree && Masked::value) unseen = !((any[q / 2] >> (16 * (q & 1) + 8 * e)) & 1u);
          if (unseen) ks = kz = vs[q][e] = vo[q][e] = 0.f;
          big = fmaxf(big, vs[q][e]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const F2 raw = fma2(sh[q][nb][e], dup(0.0625f), sl[q][nb][e]);
            F2 v = {fmaf(ks, raw.x, kz * qs[nb].x), fmaf(ks, raw.y, kz * qs[nb].y)};
            if (Masked::value) {
              if (hidden(nb, 0, q, e)) v.x = kNegInf;
              if (hidden(nb, 1, q, e)) v.y = kNegInf;
            }
            x[q][nb][e] = v;
            top[nb].x = fmaxf(top[nb].x, v.x);
            top[nb].y = fmaxf(top[nb].y, v.y);
          }
        }
      }
      bool over = big > sref;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) over = over || top[nb].x > m[nb].x + kLazy || top[nb].y > m[nb].y + kLazy;
      if (__any_sync(0xffffffffu, over)) {
        // move the references: the rows' maxima and the power of two above the values' scales
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, q));
        float ratio = 1.f;
        if (big > sref) {  // 2^(exponent + 1); warp-uniform: vs depends on g alone
          const float up = __uint_as_float(((__float_as_uint(big) >> 23) + 1) << 23);
          ratio = sref / up;
          sref = up;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int q = 4; q < 32; q <<= 1) {
            top[nb].x = fmaxf(top[nb].x, __shfl_xor_sync(0xffffffffu, top[nb].x, q));
            top[nb].y = fmaxf(top[nb].y, __shfl_xor_sync(0xffffffffu, top[nb].y, q));
          }
          const F2 nm = {fmaxf(m[nb].x, top[nb].x), fmaxf(m[nb].y, top[nb].y)};
          const F2 f = {m[nb].x == nm.x ? 1.f : ex2(m[nb].x - nm.x), m[nb].y == nm.y ? 1.f : ex2(m[nb].y - nm.y)};
          m[nb] = nm;
          l[nb] = mul2(l[nb], f);
          pz[nb] = mul2(pz[nb], f);
          const F2 fo = mul2(f, dup(ratio));
#pragma unroll
          for (int t = 0; t < CW * 2; ++t) {
            o[t][nb][0] = mul2(o[t][nb][0], fo);
            o[t][nb][1] = mul2(o[t][nb][1], fo);
          }
        }
      }
      // ---- probabilities, and O^T += V^T P^T --------------------------------------
      // -8 sum(p s) of these tokens is summed beside the codes' products, from the same halves
      // of p s, and added at their end: the running sums are those of c - 8.  (Sums of the
      // codes themselves grow with the tokens while the result does not: the tensor cores'
      // rounding towards zero left 1e-3 of it at 131,000 tokens, five times the fp16 output's
      // own rounding.)
      F2 eights[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) eights[nb][0] = eights[nb][1] = dup(0.f);
      const float rs = 64.f / sref;
#pragma unroll
      for (int q = 0; q < GI; ++q) {
        const uint8_t* sg = st + q * GR;
        uint32_t v0[CW], v1[CW];
        load_words<CW>(sg + 8 * D + lane * (D / 8), v0);
        load_words<CW>(sg + 12 * D + lane * (D / 8), v1);
        uint32_t ph[NB][2], pl[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const F2 xm = add2(x[q][nb][e], {-m[nb].x, -m[nb].y});
            const F2 pe = {ex2(xm.x), ex2(xm.y)};
            l[nb] = add2(l[nb], pe);
            const float wt = vs[q][e] * rs;
            F2 y = {pe.x * wt, pe.y * wt};
            if (!Masked::value) {
              pz[nb] = {fmaf(pe.x, vo[q][e], pz[nb].x), fmaf(pe.y, vo[q][e], pz[nb].y)};
            } else {  // a token that is masked for one row alone may have a NaN scale
              if (hidden(nb, 0, q, e)) y.x = 0.f;
              else pz[nb].x = fmaf(pe.x, vo[q][e], pz[nb].x);
              if (hidden(nb, 1, q, e)) y.y = 0.f;
              else pz[nb].y = fmaf(pe.y, vo[q][e], pz[nb].y);
            }
            const __half2 hi = __floats2half2_rn(y.x, y.y);
            const float2 back = __half22float2(hi);
            ph[nb][e] = transpose8x8(h2_bits(hi));
            pl[nb][e] = transpose8x8(h2_bits(__floats2half2_rn(y.x - back.x, y.y - back.y)));
          }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(eights[nb], kEight, kEight, kEight, kEight, ph[nb][0], ph[nb][1]);
        // two words' operands at a time, the first halves of P before the second: four products lie
        // between two that add to the same sums
#pragma unroll
        for (int j0 = 0; j0 < CW; j0 += 2) {
          uint32_t lo[2][4], hi[2][4];
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const uint32_t a0 = v0[j0 + d], a1 = v0[j0 + d] >> 8, a2 = v1[j0 + d], a3 = v1[j0 + d] >> 8;
            lo[d][0] = a0 & 0x000F000Fu; lo[d][1] = a1 & 0x000F000Fu;
            lo[d][2] = a2 & 0x000F000Fu; lo[d][3] = a3 & 0x000F000Fu;
            hi[d][0] = a0 & 0x00F000F0u; hi[d][1] = a1 & 0x00F000F0u;
            hi[d][2] = a2 & 0x00F000F0u; hi[d][3] = a3 & 0x00F000F0u;
          }
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                const uint32_t p0 = half ? pl[nb][0] : ph[nb][0], p1 = half ? pl[nb][1] : ph[nb][1];
                mma16816(o[2 * (j0 + d)][nb], lo[d][0], lo[d][1], lo[d][2], lo[d][3], p0, p1);
                mma16816(o[2 * (j0 + d) + 1][nb], hi[d][0], hi[d][1], hi[d][2], hi[d][3], p0, p1);
              }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma16816(eights[nb], kEight, kEight, kEight, kEight, pl[nb][0], pl[nb][1]);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < CW * 2; t += 2) {  // the second of two is 16 times the value
          o[t][nb][0] = add2(o[t][nb][0], eights[nb][0]);
          o[t][nb][1] = add2(o[t][nb][1], eights[nb][1]);
          o[t + 1][nb][0] = fma2(eights[nb][0], dup(16.f), o[t + 1][nb][0]);
          o[t + 1][nb][1] = fma2(eights[nb][1], dup(16.f), o[t + 1][nb][1]);
        }
    };

    for (int i = 0; i < cnt; ++i) {
      const int t0 = (w.lo + cur.g + i) * Sh::kBlock;
      const int stage = done % S;
      const uint8_t* st = ring_ptr + stage * BB;
      if (!wait_warp(smem_addr(&ctrl->full[warp * S + stage]), (uint32_t)((done / S) & 1), wc)) {
        ok = false;
        break;
      }
      // one version for blocks that every row sees whole, one with masks
#pragma unroll 1
      for (int q = 0; q < GB; q += GI) {
        const int t = t0 + q * kGranule;
        if (t + Sh::kStep <= all_hi && t >= all_lo) block(std::false_type{}, t, st + q * GR);
        else if (t < any_hi && t + Sh::kStep > any_lo) block(std::true_type{}, t, st + q * GR);
      }
      __syncwarp();
      ++done;
      if (issued < total) issue(stage);
    }
    if (!ok) break;

    // ---- the end of the segment, or of the stripe --------------------------------------
    const float unit = kCodeUnit * sref * (1.f / 64.f);
    const bool whole = cnt == w.n;
    const bool tail = cur.g != 0;  // a segment that began before: this warp's first part, else its last
    // a part goes to the ring once the stream is done, else to the workspace
    float* part = done == total ? reinterpret_cast<float*>(ring_ptr)
                                : p.firsts + (long long)(blockIdx.x * W + warp) * (Sh::kPart / 4);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int q = 4; q < 32; q <<= 1) {
        l[nb] = add2(l[nb], {__shfl_xor_sync(0xffffffffu, l[nb].x, q), __shfl_xor_sync(0xffffffffu, l[nb].y, q)});
        pz[nb] = add2(pz[nb], {__shfl_xor_sync(0xffffffffu, pz[nb].x, q), __shfl_xor_sync(0xffffffffu, pz[nb].y, q)});
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nb * 8 + 2 * c + e;
        float ll = e ? l[nb].y : l[nb].x;
        const float zz = e ? pz[nb].y : pz[nb].x;
        if (!whole && g == 0) {
          part[RB * Sh::kOStride + 2 * row] = e ? m[nb].y : m[nb].x;
          part[RB * Sh::kOStride + 2 * row + 1] = ll;
        }
        if (kTree && whole && rb * RB + row < rows) ll = kv_tree_sum(p, w.s, kv_div_group(p, rb * RB + row), ll);
#pragma unroll
        for (int j = 0; j < CW; ++j) {
          const F2 a = o[2 * j][nb][0], b = o[2 * j + 1][nb][0], d = o[2 * j][nb][1], f = o[2 * j + 1][nb][1];
          float4 v;
          v.x = fmaf(e ? a.y : a.x, unit, zz);
          v.y = fmaf(e ? b.y : b.x, unit * 0.0625f, zz);
          v.z = fmaf(e ? d.y : d.x, unit, zz);
          v.w = fmaf(e ? f.y : f.x, unit * 0.0625f, zz);
          if (!whole)
            *reinterpret_cast<float4*>(part + row * Sh::kOStride + g * (D / 8) + 4 * j) = v;
          else if (rb * RB + row < rows)
            store_row<kTree>(p, w.s, h, rb * RB + row, g * (D / 8) + 4 * j, D, v, ll);
        }
      }
    }
    if (!whole && lane == 0) {
      Parts& q = ctrl->parts[warp];
      if (tail) {
        q.first = 1;
        q.first_ends = cur.g + cnt == w.n;
        q.first_last = done == total;
      } else {
        q.last = 1;
      }
      q.seg[tail ? 0 : 1] = {w.s, h, rb, w.n, Sh::kStart ? from : from + done - cnt - cur.g};
    }
    if constexpr (Sh::kStart > 0) from += w.n + Sh::kStart;
    advance<Sh>(p, cur, cnt);
  }
  // nothing may still be in flight into this CTA's shared memory
  for (; done < issued; ++done)
    if (lane == 0) wait_drain(smem_addr(&ctrl->full[warp * S + done % S]), (uint32_t)((done / S) & 1), wc);
  __syncthreads();
  if (ctrl->abort) return;

  // ---- segments cut between warps: runs of parts of consecutive warps ------------------
  // A run begins with a warp's last part, or with the first part of the CTA's
  // first warp that has any blocks (a segment that began in an earlier CTA), and
  // goes on with the next warps' first parts until the segment ends.  Lane 0
  // looks at the run that began before, lane 1 + q at the one that warp q begins.
  constexpr int kVec = RB * D / 4;  // a thread joins four channels of one row
  int run_q0 = 0, run_end = 0, run_ends = 0, run_on = 0;
  {
    int q = lane - 1;
    if (lane == 0)
      for (q = 0; q < W - 1 && ctrl->parts[q].idle;) ++q;
    if (q < W) {
      run_on = lane ? ctrl->parts[q].last : ctrl->parts[q].first;
      run_ends = lane == 0 && ctrl->parts[q].first_ends;
      run_q0 = q;
      for (run_end = q + 1; run_on && !run_ends && run_end < W; ++run_end) {
        const Parts& next = ctrl->parts[run_end];
        if (!next.idle && !next.first) break;
        run_ends = !next.idle && next.first_ends;
      }
    }
  }
  const uint32_t runs = __ballot_sync(0xffffffffu, run_on);
  // the (at most two) runs whose segments other CTAs share: that of lane 0, and
  // the last one if its segment goes on
  const uint32_t shared = runs & ~__ballot_sync(0xffffffffu, lane != 0 && run_ends);
  for (int v = tid; v < __popc(runs) * kVec; v += W * 32) {
    const int lead = (int)__fns(runs, 0, v / kVec + 1);  // the same for the whole warp
    const int q0 = __shfl_sync(0xffffffffu, run_q0, lead), end = __shfl_sync(0xffffffffu, run_end, lead);
    const Segment& sg = ctrl->parts[q0].seg[lead != 0];
    const int row = (v % kVec) / (D / 4), ch = (v % (D / 4)) * 4;
    // all parts' loads first, then the sums in order
    float2 pml[W];
    float4 pa[W];
#pragma unroll
    for (int q = 0; q < W; ++q) {
      pml[q] = make_float2(kLowest, 0.f);
      pa[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q >= q0 && q < end && !ctrl->parts[q].idle) {
        const bool in_ring = (lead != 0 && q == q0) || ctrl->parts[q].first_last;
        const float* at = in_ring ? reinterpret_cast<const float*>(smem + Sh::kRing + q * (S * BB))
                                  : p.firsts + (long long)(blockIdx.x * W + q) * (Sh::kPart / 4);
        pml[q] = *reinterpret_cast<const float2*>(at + RB * Sh::kOStride + 2 * row);
        pa[q] = *reinterpret_cast<const float4*>(at + row * Sh::kOStride + ch);
      }
    }
    float top = kLowest, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < W; ++q) join(pml[q], pa[q], top, sum, acc);
    if ((shared >> lead) & 1u) {
      float* part = p.partials + (2ll * blockIdx.x + (lead != 0)) * (RB * (D + 2));
      __stcg(reinterpret_cast<float4*>(part + row * D + ch), acc);
      if (ch == 0) __stcg(reinterpret_cast<float2*>(part + RB * D + 2 * row), make_float2(top, sum));
    } else if (sg.rb * RB + row < sg.s.nq * p.group) {
      if (kTree) sum = kv_tree_sum(p, sg.s, kv_div_group(p, sg.rb * RB + row), sum);
      store_row<kTree>(p, sg.s, sg.h, sg.rb * RB + row, ch, D, acc, sum);
    }
  }
  if (shared == 0) return;

  // ---- segments cut between CTAs: the last to arrive joins the parts in stripe order ---
  // k = 0: the one that began before, k = 1: the one that goes on
  const bool on[2] = {(shared & 1u) != 0, (shared & ~1u) != 0};
  const int goes_on = 31 - __clz((int)(shared | 1u));
  const Segment* seg[2] = {&ctrl->parts[__shfl_sync(0xffffffffu, run_q0, 0)].seg[0],
                           &ctrl->parts[__shfl_sync(0xffffffffu, run_q0, goes_on)].seg[1]};
  int c0[2] = {0, 0}, c1[2] = {0, 0};  // the CTAs that share it
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (on[k]) {
      c0[k] = (int)owner_of(seg[k]->s0 + Sh::kStart, U, G);
      c1[k] = (int)owner_of(seg[k]->s0 + Sh::kStart + seg[k]->n - 1, U, G);
    }
  __syncthreads();
  if (tid < 2 && on[tid]) {
    const int first_cta = tid ? c0[1] : c0[0], last_cta = tid ? c1[1] : c1[0];
    // release and acquire at the card's scope, for the whole CTA by way of the barriers
    int arrived;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(arrived) : "l"(p.counters + first_cta) : "memory");
    ctrl->arrived[tid] = arrived == last_cta - first_cta;
    if (arrived == last_cta - first_cta) p.counters[first_cta] = 0;  // all are here: ready for the next call
    __threadfence();
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!on[k] || !ctrl->arrived[k]) continue;
    const Segment sg = *seg[k];
    for (int v = tid; v < kVec; v += W * 32) {
      const int row = v / (D / 4), ch = (v - row * (D / 4)) * 4;
      if (sg.rb * RB + row >= sg.s.nq * p.group) continue;
      float top = kLowest, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int kAhead = 8;  // parts loaded together
      for (int q0 = c0[k]; q0 <= c1[k]; q0 += kAhead) {
        float2 ml[kAhead];
        float4 a[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          ml[i] = make_float2(kLowest, 0.f);
          a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (q0 + i <= c1[k]) {  // the first CTA's part is in its slot 1, the others' in slot 0
            const float* src = p.partials + (2ll * (q0 + i) + (q0 + i == c0[k] ? 1 : 0)) * (RB * (D + 2));
            ml[i] = __ldcg(reinterpret_cast<const float2*>(src + RB * D + 2 * row));
            a[i] = __ldcg(reinterpret_cast<const float4*>(src + row * D + ch));
          }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) join(ml[i], a[i], top, sum, acc);
      }
      if (kTree) sum = kv_tree_sum(p, sg.s, kv_div_group(p, sg.rb * RB + row), sum);
      store_row<kTree>(p, sg.s, sg.h, sg.rb * RB + row, ch, D, acc, sum);
    }
  }
}

template <int D, int NB, bool kTree>
cudaError_t launch(const KvAttnParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Shape<D, NB, kTree>::W * 32);
  cfg.dynamicSmemBytes = Shape<D, NB, kTree>::kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attn_kernel<D, NB, kTree>, p);
}

}  // namespace

cudaError_t kv_attn_set_smem_limit() {
  cudaError_t e = cudaSuccess;
#define W4A16_SET(D, NB, T)                                                                                   \
  if (e == cudaSuccess)                                                                                       \
    e = cudaFuncSetAttribute(kv_attn_kernel<D, NB, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, NB, T>::kSmem);
  W4A16_SET(128, 1, false) W4A16_SET(128, 2, false) W4A16_SET(64, 1, false) W4A16_SET(64, 2, false)
  W4A16_SET(128, 1, true) W4A16_SET(128, 2, true) W4A16_SET(64, 1, true) W4A16_SET(64, 2, true)
#undef W4A16_SET
  return e;
}

template <bool kTree>
static cudaError_t launch_shape(const KvAttnParams& p, int D, int nb, int grid, cudaStream_t stream) {
  if (D == 128) return nb == 1 ? launch<128, 1, kTree>(p, grid, stream) : launch<128, 2, kTree>(p, grid, stream);
  return nb == 1 ? launch<64, 1, kTree>(p, grid, stream) : launch<64, 2, kTree>(p, grid, stream);
}

cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int nb, int grid, cudaStream_t stream) {
  return p.tree ? launch_shape<true>(p, D, nb, grid, stream) : launch_shape<false>(p, D, nb, grid, stream);
}

}  // namespace w4a16
