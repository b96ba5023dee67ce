// kv_attn.cu -- causal attention of new tokens over the 4-bit paged cache, for
// few query rows per key head (single tokens, a few proposed ones):
//     O[i][h] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q[i][h] . k_t - max),
// over the cached tokens t <= position(i) (and t > position(i) - window).
//
// Bound: streaming the cache, 2 (D/2 + 4) bytes per token and key head, once.
//   * The work is (request, key head, block of 8 NB query rows) segments of
//     16-token granules; the rows of a block are the G query heads that share
//     the key head, for one or more query tokens, so that a granule is read
//     once for all of them.  Every CTA (one per SM) takes an equal contiguous
//     stripe of granules, found on the device from the lengths.
//   * Its W warps take granules in turn, each with its own ring of bulk copies
//     (one per granule), its own running maximum, sum and accumulators: no
//     barrier inside a segment.
//   * Both products run on mma.sync with the cache as the 16-row operand and the
//     query rows as the 8 columns: S^T[16 tokens x 8 rows] = K Q^T and
//     O^T[16 channels x 8 rows] += V^T P^T.  A code c is fed as the fp16
//     subnormal c * 2^-24 (one AND per pair; the nibble four bits up is
//     16 c * 2^-24): the products are exact and scales, offsets and the powers
//     of two are applied to the fp32 results (kv.cuh has the algebra).
//   * p_t s_t is fed as the sum of two fp16 numbers (22 bits): with one, the
//     rounding of the probabilities times uncentred codes would be three times
//     the rounding of the fp16 output.  s_t is normalised by a running power of
//     two so that neither half falls below fp16's range.
//   * The maximum is only moved when a score exceeds it by 2^8 (one vote per
//     granule instead of shuffles and a rescaling).
// A segment cut by stripe boundaries is finished by whichever of its CTAs
// arrives last, summing all parts in stripe order (so the result does not
// depend on the order of arrival).  Nothing waits for another CTA.
#include "kv.cuh"

namespace w4a16 {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kLazy = 8.f;            // log2 of how far a score may exceed the reference
constexpr float kCodeUnit = 16777216.f;  // 2^24: an fp16 subnormal's unit is 2^-24
constexpr float kMinSref = 9.313225746154785e-10f;  // 2^-30

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = lds128(addr);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  }
}

// Four channels of an output row: row rr of key head h, normalised.  A row
// that sees no token is zero.
__device__ __forceinline__ void store_row(const KvAttnParams& p, const KvSeq& s, int h, int rr, int ch, int D,
                                          float4 acc, float sum) {
  const int i = rr / p.group, head = h * p.group + rr - i * p.group;
  const float inv = s.len - s.nq + i >= 0 ? 1.f / sum : 0.f;
  if (inv == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);
  uint2 v;
  v.x = h2_bits(__floats2half2_rn(acc.x * inv, acc.y * inv));
  v.y = h2_bits(__floats2half2_rn(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(p.out + ((long long)(s.q0 + i) * p.heads + head) * D + ch) = v;
}

// One request's share of the work: its granules [g_lo, g_lo + n) and the
// number of its blocks of query rows.
struct SeqWork {
  KvSeq s;
  int g_lo, n, rbs;
};

template <int RB>
__device__ __forceinline__ SeqWork seq_work(const KvAttnParams& p, int b, bool report) {
  SeqWork w;
  w.s = kv_seq(p.kv, b, report);
  if (w.s.nq > w.s.len && report) kv_fail(p.kv, kKvSiteLen);
  const int rows = w.s.nq * p.group;
  w.rbs = rows > p.max_rows ? 0 : (rows + RB - 1) / RB;
  const int first = w.s.len - w.s.nq;  // position of the first query token
  const int lo = p.window > 0 ? max(0, first - p.window + 1) : 0;
  w.g_lo = lo >> 4;
  w.n = max(1, ((w.s.len + 15) >> 4) - w.g_lo);
  return w;
}

// A place in the stripe: granule g of segment seg (key head * rbs + row block)
// of request b.
struct Cursor {
  int b, seg, g;
  SeqWork w;
};

template <int RB>
__device__ __forceinline__ void advance(const KvAttnParams& p, Cursor& c, int by) {
  c.g += by;
  while (c.g >= c.w.n) {
    c.g -= c.w.n;
    if (++c.seg == p.kv.hkv * c.w.rbs) {
      c.seg = 0;
      do {
        if (++c.b >= p.kv.B) { c.g = 0; return; }
        c.w = seq_work<RB>(p, c.b, false);
      } while (c.w.rbs == 0);
    }
  }
}

// Largest W that the shared memory of an SM holds with a useful ring.
template <int D, int NB>
struct Shape {
  static constexpr int W = NB == 1 ? 16 : 8;    // warps
  static constexpr int S = NB == 1 ? 4 : 8;     // granules in a warp's ring
  static constexpr int RB = 8 * NB;             // query rows
  static constexpr int GR = kv_granule_bytes(D);
  static constexpr int kOStride = D + 4;        // floats of a row in the merge buffer
  static constexpr int kRing = 1024;
  static constexpr int kMerge = kRing + W * S * GR;
  static constexpr int kMl = kMerge + W * RB * kOStride * 4;
  static constexpr int kSmem = kMl + W * RB * 2 * 4;
};

struct AttnCtrl {
  uint64_t full[64];       // [W][S]
  long long scan[16];
  long long total;
  long long start_off;     // first unit's offset in its request
  int start_b;
  int abort;
  int last;
};
static_assert(sizeof(AttnCtrl) <= 1024, "control block too large");

template <int D, int NB>
__global__ void __launch_bounds__(Shape<D, NB>::W * 32, 1) kv_attn_kernel(const KvAttnParams p) {
  using Sh = Shape<D, NB>;
  constexpr int W = Sh::W, S = Sh::S, RB = Sh::RB, GR = Sh::GR, CW = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  AttnCtrl* ctrl = reinterpret_cast<AttnCtrl*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_addr(smem) + Sh::kRing + warp * (S * GR);
  float* const merge = reinterpret_cast<float*>(smem + Sh::kMerge);
  float* const ml = reinterpret_cast<float*>(smem + Sh::kMl);

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(smem_addr(&ctrl->full[warp * S + s]), 1);
    if (warp == 0) {
      ctrl->abort = 0;
      ctrl->start_b = -1;
    }
    fence_mbarrier_init();
  }
  if (tid == 0) griddep_launch_dependents();
  griddep_wait();

  // ---- this CTA's stripe of granules -----------------------------------------
  const int per = (p.kv.B + W * 32 - 1) / (W * 32);
  const int b0 = min(tid * per, p.kv.B), b1 = min(b0 + per, p.kv.B);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqWork w = seq_work<RB>(p, b, blockIdx.x == 0);
    mine += (long long)p.kv.hkv * w.rbs * w.n;
  }
  long long before = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, before, m);
    if (lane >= m) before += o;
  }
  if (lane == 31) ctrl->scan[warp] = before;
  __syncthreads();
  long long U = 0, base = 0;
  for (int w = 0; w < W; ++w) {
    if (w == warp) base = U;
    U += ctrl->scan[w];
  }
  before += base - mine;
  if (U == 0) return;
  // small problems: at least a granule per warp for every CTA that takes part
  const long long G = min((long long)gridDim.x, (U + W - 1) / W);
  if (blockIdx.x >= G) return;
  const long long u_begin = stripe_begin(blockIdx.x, U, G), u_end = stripe_begin(blockIdx.x + 1, U, G);
  if (u_begin >= before && u_begin < before + mine) {
    long long off = u_begin - before;
    for (int b = b0; b < b1; ++b) {
      const SeqWork w = seq_work<RB>(p, b, false);
      const long long n = (long long)p.kv.hkv * w.rbs * w.n;
      if (off < n) {
        ctrl->start_b = b;
        ctrl->start_off = off;
        break;
      }
      off -= n;
    }
  }
  __syncthreads();
  Cursor cur;
  cur.b = ctrl->start_b;
  cur.w = seq_work<RB>(p, cur.b, false);
  cur.seg = (int)(ctrl->start_off / cur.w.n);
  cur.g = (int)(ctrl->start_off - (long long)cur.seg * cur.w.n);

  const WaitCtx wc{&ctrl->abort, p.kv.status, p.timeout_ns};
  const int total = (int)(u_end - u_begin);
  const int mine_n = total > warp ? (total - warp + W - 1) / W : 0;  // this warp's granules: warp, warp + W, ...

  // ---- the ring's producer (all lanes keep the cursor, lane 0 copies) ------------
  Cursor pc = cur;
  advance<RB>(p, pc, warp);
  int issued = 0;
  auto page_of = [&](const Cursor& k) {
    return p.kv.table[(long long)k.b * p.kv.max_pages + kv_div_page(p.kv, k.w.g_lo + k.g)];
  };
  int next_page = 0;
  if (mine_n > 0 && pc.w.s.len > 0) next_page = page_of(pc);
  auto issue = [&](int stage) {  // copies the granule at pc and moves on
    const int gi = pc.w.g_lo + pc.g;
    const bool inside = gi * kGranule < pc.w.s.len;  // else nothing is cached there (an empty request)
    const bool ok = next_page >= 0 && next_page < p.kv.n_pages;
    const uint32_t bar = smem_addr(&ctrl->full[warp * S + stage]);
    if (lane == 0) {
      if (inside && ok) {
        const int h = pc.seg / pc.w.rbs;
        mbar_arrive_expect_tx(bar, GR);
        bulk_g2s(ring + stage * GR,
                 p.kv.cache + next_page * p.kv.page_bytes + h * p.kv.head_bytes +
                     (long long)(gi - kv_div_page(p.kv, gi) * p.kv.page16) * GR,
                 GR, bar, policy_evict_first());
      } else {
        if (inside) kv_fail(p.kv, kKvSitePage);
        mbar_arrive(bar);  // no copy: nobody sees the granule, or its page is reported as missing
      }
    }
    ++issued;
    if (issued < mine_n) {
      advance<RB>(p, pc, W);
      if (pc.w.s.len > 0) next_page = page_of(pc);
    }
  };
  while (issued < min(S, mine_n)) issue(issued);

  int done = 0;  // granules of this warp consumed
  int u = 0;     // units of the stripe passed
  while (u < total) {
    const SeqWork& w = cur.w;
    const int cnt = min(total - u, w.n - cur.g);
    const int h = cur.seg / w.rbs, rb = cur.seg - h * w.rbs;
    const int rows = w.s.nq * p.group;
    const int first = w.s.len - w.s.nq;

    // ---- queries: B operands in the channel order of the codes, and their sums ----
    uint32_t qf[NB][CW * 4];
    float qs[NB][2];
    int hi_pos[NB][2], lo_pos[NB][2];  // tokens seen by rows 2c, 2c + 1: [lo, hi)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int row = rb * RB + nb * 8 + g;
      float sum = 0.f;
      if (row < rows) {
        const int i = row / p.group, head = h * p.group + row - i * p.group;
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
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[nb][e] = __shfl_sync(0xffffffffu, sum, (2 * c + e) * 4) * p.scale_log2;
        const int rr = rb * RB + nb * 8 + 2 * c + e;
        const int pos = first + rr / p.group;
        hi_pos[nb][e] = rr < rows ? pos + 1 : 0;
        lo_pos[nb][e] = p.window > 0 ? pos - p.window + 1 : 0;
      }
    }
    // tokens every row sees, [all_lo, all_hi), and tokens any row sees
    const int i_first = rb * RB / p.group, i_last = (min(rows, (rb + 1) * RB) - 1) / p.group;
    const int all_hi = first + i_first + 1, any_hi = first + i_last + 1;
    const int all_lo = p.window > 0 ? first + i_last - p.window + 1 : 0;
    const int any_lo = p.window > 0 ? first + i_first - p.window + 1 : 0;

    float m[NB][2], l[NB][2], pz[NB][2], o[CW * 2][NB][4];
    float sref = kMinSref, rs = 64.f / kMinSref;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nb][e] = kNegInf;
        l[nb][e] = pz[nb][e] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < CW * 2; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][nb][k] = 0.f;
    }

    // this warp's granules of the segment: units u + x with (u + x) % W == warp
    for (int x = (warp - u % W + W) % W; x < cnt; x += W) {
      const int t0 = (w.g_lo + cur.g + x) * kGranule;
      const int stage = done % S;
      const uint32_t st = ring + stage * GR;
      const uint32_t ph = (uint32_t)((done / S) & 1);
      if (!wait_warp(smem_addr(&ctrl->full[warp * S + stage]), ph, wc)) break;
      uint32_t k0[CW], k1[CW], v0[CW], v1[CW];
      lds_words<CW>(st + g * (D / 2) + c * (D / 8), k0);
      lds_words<CW>(st + (g + 8) * (D / 2) + c * (D / 8), k1);
      lds_words<CW>(st + 8 * D + lane * (D / 8), v0);
      lds_words<CW>(st + 12 * D + lane * (D / 8), v1);
      uint32_t pa[2], pb[2];
      lds_words<2>(st + 16 * D + g * 8, pa);
      lds_words<2>(st + 16 * D + (g + 8) * 8, pb);
      __syncwarp();
      ++done;
      if (issued < mine_n) issue(stage);
      if (t0 >= any_hi || t0 + kGranule <= any_lo) continue;
      const bool full = t0 + kGranule <= all_hi && t0 >= all_lo;

      // scales and offsets of tokens g (index 0) and g + 8 (1); nothing is
      // taken from slots that no row sees (they may hold anything)
      float ks[2], kz[2], vs[2], vz[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t* pr = e ? pb : pa;
        const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&pr[0]));
        const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&pr[1]));
        const int t = t0 + g + 8 * e;
        const bool seen = full || (t < any_hi && t >= any_lo);
        ks[e] = seen ? kf.x * (kCodeUnit * p.scale_log2) : 0.f;
        kz[e] = seen ? kf.y - 8.f * kf.x : 0.f;
        vs[e] = seen ? vf.x : 0.f;
        vz[e] = seen ? vf.y - 8.f * vf.x : 0.f;
      }

      // ---- S^T = K Q^T on the codes: low nibbles and high (x 16) apart -----------
      float sl[NB][4], sh[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) sl[nb][k] = sh[nb][k] = 0.f;
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const uint32_t a0 = k0[j], a1 = k1[j], a2 = k0[j] >> 8, a3 = k1[j] >> 8;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          mma16816(sl[nb], a0 & 0x000F000Fu, a1 & 0x000F000Fu, a2 & 0x000F000Fu, a3 & 0x000F000Fu,
                   qf[nb][4 * j], qf[nb][4 * j + 1]);
          mma16816(sh[nb], a0 & 0x00F000F0u, a1 & 0x00F000F0u, a2 & 0x00F000F0u, a3 & 0x00F000F0u,
                   qf[nb][4 * j + 2], qf[nb][4 * j + 3]);
        }
      }
      // scores in units of log2: element k is token g + 8 (k >> 1), row 2c + (k & 1)
      bool over = vs[0] > sref || vs[1] > sref;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tt = k >> 1, e = k & 1;
          const float raw = fmaf(sh[nb][k], 0.0625f, sl[nb][k]);
          float xs = fmaf(ks[tt], raw, kz[tt] * qs[nb][e]);
          if (!full) {
            const int t = t0 + g + 8 * tt;
            if (t >= hi_pos[nb][e] || t < lo_pos[nb][e]) xs = kNegInf;
          }
          sl[nb][k] = xs;
          over = over || xs > m[nb][e] + kLazy;
        }
      if (__any_sync(0xffffffffu, over)) {
        // move the references: the rows' maxima and the power of two above the values' scales
        float sm = fmaxf(vs[0], vs[1]);
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) sm = fmaxf(sm, __shfl_xor_sync(0xffffffffu, sm, q));
        float ratio = 1.f;
        if (sm > sref) {  // 2^(exponent + 1); warp-uniform: vs depends on g alone
          const float up = __uint_as_float(((__float_as_uint(sm) >> 23) + 1) << 23);
          ratio = sref / up;
          sref = up;
          rs = 64.f / up;
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(sl[nb][e], sl[nb][2 + e]);
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, q));
            top = fmaxf(top, m[nb][e]);
            const float f = m[nb][e] == top ? 1.f : ex2(m[nb][e] - top);
            m[nb][e] = top;
            l[nb][e] *= f;
            pz[nb][e] *= f;
            const float fo = f * ratio;
#pragma unroll
            for (int t = 0; t < CW * 2; ++t) {
              o[t][nb][e] *= fo;
              o[t][nb][2 + e] *= fo;
            }
          }
      }
      // ---- probabilities; P^T's operand halves ------------------------------------
      uint32_t ph0[NB], ph1[NB], pl0[NB], pl1[NB];
      const float w0 = vs[0] * rs, w1 = vs[1] * rs;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tt = k >> 1, e = k & 1;
          const float ref = m[nb][e] == kNegInf ? 0.f : m[nb][e];
          const float pe = ex2(sl[nb][k] - ref);
          l[nb][e] += pe;
          float zz = pe * vz[tt];
          y[k] = pe * (tt ? w1 : w0);
          if (!full) {  // a masked token's scale may be NaN
            const int t = t0 + g + 8 * tt;
            if (t >= hi_pos[nb][e] || t < lo_pos[nb][e]) zz = y[k] = 0.f;
          }
          pz[nb][e] += zz;
        }
        const __half2 h0 = __floats2half2_rn(y[0], y[1]), h1 = __floats2half2_rn(y[2], y[3]);
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        ph0[nb] = transpose8x8(h2_bits(h0));
        ph1[nb] = transpose8x8(h2_bits(h1));
        pl0[nb] = transpose8x8(h2_bits(__floats2half2_rn(y[0] - f0.x, y[1] - f0.y)));
        pl1[nb] = transpose8x8(h2_bits(__floats2half2_rn(y[2] - f1.x, y[3] - f1.y)));
      }
      // ---- O^T += V^T P^T -----------------------------------------------------------
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const uint32_t a0 = v0[j], a1 = v0[j] >> 8, a2 = v1[j], a3 = v1[j] >> 8;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const uint32_t l0 = a0 & 0x000F000Fu, l1 = a1 & 0x000F000Fu, l2 = a2 & 0x000F000Fu, l3 = a3 & 0x000F000Fu;
          const uint32_t h0 = a0 & 0x00F000F0u, h1 = a1 & 0x00F000F0u, h2 = a2 & 0x00F000F0u, h3 = a3 & 0x00F000F0u;
          mma16816(o[2 * j][nb], l0, l1, l2, l3, ph0[nb], ph1[nb]);
          mma16816(o[2 * j + 1][nb], h0, h1, h2, h3, ph0[nb], ph1[nb]);
          mma16816(o[2 * j][nb], l0, l1, l2, l3, pl0[nb], pl1[nb]);
          mma16816(o[2 * j + 1][nb], h0, h1, h2, h3, pl0[nb], pl1[nb]);
        }
      }
    }

    // ---- the warps' parts -> shared memory -------------------------------------------
    const float unit = kCodeUnit * sref * (1.f / 64.f);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) {
          l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], q);
          pz[nb][e] += __shfl_xor_sync(0xffffffffu, pz[nb][e], q);
        }
        const int row = nb * 8 + 2 * c + e;
        if (g == 0) {
          ml[(warp * RB + row) * 2] = m[nb][e];
          ml[(warp * RB + row) * 2 + 1] = l[nb][e];
        }
        float* dst = merge + (warp * RB + row) * Sh::kOStride + g * (D / 8);
#pragma unroll
        for (int j = 0; j < CW; ++j) {
          float4 v;
          v.x = fmaf(o[2 * j][nb][e], unit, pz[nb][e]);
          v.y = fmaf(o[2 * j + 1][nb][e], unit * 0.0625f, pz[nb][e]);
          v.z = fmaf(o[2 * j][nb][2 + e], unit, pz[nb][e]);
          v.w = fmaf(o[2 * j + 1][nb][2 + e], unit * 0.0625f, pz[nb][e]);
          *reinterpret_cast<float4*>(dst + 4 * j) = v;
        }
      }
    __syncthreads();

    // ---- the CTA's part; whole segments are finished, others published ---------------
    const bool whole = cnt == w.n;
    const long long s0 = u_begin + u - cur.g;  // the segment's first unit
    const int slot = 2 * blockIdx.x + (cur.g == 0 ? 1 : 0);
    float* part = p.partials + (long long)slot * (RB * (D + 2));
    constexpr int kVec = RB * D / 4;
    for (int v = tid; v < kVec; v += W * 32) {
      const int row = v / (D / 4), ch = (v - row * (D / 4)) * 4;
      float top = kNegInf;
#pragma unroll
      for (int q = 0; q < W; ++q) top = fmaxf(top, ml[(q * RB + row) * 2]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float mq = ml[(q * RB + row) * 2], lq = ml[(q * RB + row) * 2 + 1];
        if (lq == 0.f) continue;
        const float f = mq == top ? 1.f : ex2(mq - top);
        const float4 a = *reinterpret_cast<const float4*>(merge + (q * RB + row) * Sh::kOStride + ch);
        sum = fmaf(lq, f, sum);
        acc.x = fmaf(a.x, f, acc.x);
        acc.y = fmaf(a.y, f, acc.y);
        acc.z = fmaf(a.z, f, acc.z);
        acc.w = fmaf(a.w, f, acc.w);
      }
      if (whole) {
        const int rr = rb * RB + row;
        if (rr < rows) store_row(p, w.s, h, rr, ch, D, acc, sum);
      } else {
        __stcg(reinterpret_cast<float4*>(part + row * D + ch), acc);
        if (ch == 0) {
          __stcg(part + RB * D + 2 * row, top);
          __stcg(part + RB * D + 2 * row + 1, sum);
        }
      }
    }
    if (!whole) {
      const long long c0 = stripe_owner(s0, U, G), c1 = stripe_owner(s0 + w.n - 1, U, G);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        int* counter = p.counters + c0;
        const int arrived = atomicAdd(counter, 1);
        ctrl->last = arrived == (int)(c1 - c0);
        if (ctrl->last) *counter = 0;  // everyone has arrived: ready for the next call
        __threadfence();
      }
      __syncthreads();
      if (ctrl->last) {
        for (int v = tid; v < kVec; v += W * 32) {
          const int row = v / (D / 4), ch = (v - row * (D / 4)) * 4;
          const int rr = rb * RB + row;
          if (rr >= rows) continue;
          // the parts in stripe order: the first CTA's is its last segment's (slot
          // 1), the others' their first (slot 0)
          float top = kNegInf, sum = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (long long q = c0; q <= c1; ++q) {
            const float* src = p.partials + (2 * q + (q == c0 ? 1 : 0)) * (RB * (D + 2));
            const float mq = __ldcg(src + RB * D + 2 * row), lq = __ldcg(src + RB * D + 2 * row + 1);
            const float4 a = __ldcg(reinterpret_cast<const float4*>(src + row * D + ch));
            if (lq == 0.f) continue;
            const float nt = fmaxf(top, mq);
            const float fo = top == nt ? 1.f : ex2(top - nt), fn = mq == nt ? 1.f : ex2(mq - nt);
            top = nt;
            sum = fmaf(sum, fo, lq * fn);
            acc.x = fmaf(acc.x, fo, a.x * fn);
            acc.y = fmaf(acc.y, fo, a.y * fn);
            acc.z = fmaf(acc.z, fo, a.z * fn);
            acc.w = fmaf(acc.w, fo, a.w * fn);
          }
          store_row(p, w.s, h, rr, ch, D, acc, sum);
        }
      }
    }
    __syncthreads();  // the merge buffer is free again
    u += cnt;
    advance<RB>(p, cur, cnt);
  }
  // nothing may still be in flight into this CTA's shared memory
  for (; done < issued; ++done)
    if (lane == 0) wait_drain(smem_addr(&ctrl->full[warp * S + done % S]), (uint32_t)((done / S) & 1), wc);
}

template <int D, int NB>
cudaError_t launch(const KvAttnParams& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Shape<D, NB>::W * 32);
  cfg.dynamicSmemBytes = Shape<D, NB>::kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attn_kernel<D, NB>, p);
}

}  // namespace

cudaError_t kv_attn_set_smem_limit() {
  cudaError_t e = cudaSuccess;
#define W4A16_SET(D, NB)                                                                                        \
  if (e == cudaSuccess)                                                                                         \
    e = cudaFuncSetAttribute(kv_attn_kernel<D, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D, NB>::kSmem);
  W4A16_SET(128, 1) W4A16_SET(128, 2) W4A16_SET(64, 1) W4A16_SET(64, 2)
#undef W4A16_SET
  return e;
}

cudaError_t launch_kv_attn(const KvAttnParams& p, int D, int nb, int grid, cudaStream_t stream) {
  if (D == 128) return nb == 1 ? launch<128, 1>(p, grid, stream) : launch<128, 2>(p, grid, stream);
  return nb == 1 ? launch<64, 1>(p, grid, stream) : launch<64, 2>(p, grid, stream);
}

}  // namespace w4a16
