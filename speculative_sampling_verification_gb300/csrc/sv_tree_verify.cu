// Verification of a tree of drafted tokens (spec_verify_tree): the modified
// rejection sampling of "Accelerating Large Language Model Decoding with
// Speculative Sampling" (wikillm.com paper card, §4.2) with several candidates
// at a node, tried in turn.
//
// At the current node, with target row q and draft row p (softmax at
// temperature T), the children are tried in index order against the residual
// r, which is q at first. Child c of token x is accepted when
// u_c < min(1, r(x)/p(x)); a rejection turns r into max(0, r - p)/sum. The children
// are drawn from the same p, so after any number of rejections
//     r = max(0, A q - B p)
// with two scalars: max(0, max(0, A q - B p) - p) = max(0, A q - (B + 1) p),
// because where the inner maximum is 0 the outer one is too. So a rejection
// costs one pass over two rows for Z = sum max(0, A q - (B + 1) p), then
// (A, B) <- (A, B + 1) / Z, and no residual is ever stored. A sum below 2^-30 (r
// equals p but for rounding: such a rejection has that probability) leaves r
// as it was. Where q and p are equal but not their logits, A q - B p is what the
// exponentials' errors leave, up to 1.5e-10 (2^-32.6) with the short ones: at 2^-40 that was
// taken for a residual, and the next child's ratio was noise.
//
// One thread-block cluster a sequence; the vocabulary is cut into one region
// per warp of the cluster. Only the rows of visited nodes are read: from HBM
// once, then from L2. A pass ends with the warps' sums joined in a fixed order:
// within a CTA through shared memory, across the cluster by pushing each CTA's
// figures to every other, so that each CTA comes to the same decision by itself.
// The draw needs no pass of its own: the sums of the pass that made the
// residual lead to one warp's region, which that warp scans.
//
// Precision: an acceptance test goes wrong with the probability of its ratio's
// error, so the rows' sums for the tests are taken in fp32 with hardware exponentials
// (about 1e-7). A draw goes wrong when u falls between the two places of any of V
// borders, so what a draw uses (the residual's two sums and its own weights, or
// the last row's weights) is computed in float-floats with exponentials of 1e-12, in
// a pass that is made only when a node has a rejection or a draw.
//
// 64 trees of 16 nodes over 128256 tokens, bf16: 148 us, where reading the rows once takes 10. The
// dependent passes of a path bound it and sequences differ in length: 44 % of the issue
// slots are active on average, 74 % on the busiest SM. 512 threads a CTA, two an SM: 162.
// CTAs of 256 an SM, before the rows' statistics took one pass: three 193, four 164, five 169. One tree of nine nodes over 32000 tokens: 34 to 36 us.
// 64 trees over 50257 tokens (rows off 16 bytes, element loads): 111 us, over 50256 88 us.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace tvf {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;  // the portable cluster size
constexpr int kTreeMax = 128;
constexpr double kResidualMin = 9.313225746154785e-10;  // 2^-30
constexpr int kStep = 256;      // elements a warp takes at once: eight a lane

struct Args {
  const void *target, *draft;
  const int32_t *draft_index, *tokens, *parents;
  const float* uniforms;
  int32_t *out_tokens, *out_nodes, *n_acc;
  unsigned* status;
  int B, T, V, R, region;  // region: elements of a warp, a multiple of 8
  float ih, il;            // 1/T as a float-float
  float c2;                // log2(e)/T
  int unit_t;
  // The short exponentials (exp_draw2): its constants, the bound of a logit that they
  // take, and whether the temperature allows them.
  DrawConst dc;
  float reach;
  double inv_t;
  int short_ok;
};

struct Exchange {
  alignas(8) ff sum[2][kMaxCluster];  // per CTA: of q and p, or of the residual
  float top[2][kMaxCluster];   // per CTA: row maxima
};

struct Shared {
  float2 tab[256], tab1k[1024];
  Exchange x[2];
  ff wsum[2][2][kWarps];      // [buffer][q or p][warp]: sums of the warps' regions
  float wfast[2][kWarps];     // the tests' sums
  float wtop[2][kWarps];
  ff cta_sum[2][kMaxCluster];  // [buffer]: the CTAs' sums of the current residual
  double ratio[kTreeMax];  // q(x)/p(x) of the children's tokens
  int parents[kTreeMax], tokens[kTreeMax], drow[kTreeMax];
  float u[kTreeMax];
  int path[kTreeMax];
  float m[2];
  double S[2];
  // The deciding warp's word to the others: the next node, kDraw, or kResidual (a pass for a
  // new residual with these scalars; `keep` of the last one).
  int next;
  ff a, b;
  int keep;
  unsigned failure;
};

constexpr int kDraw = -1, kResidual = -2;

constexpr double kLn2 = 0.69314718055994530942;

// exp(v) for |v| of a few, to about 1e-12.
SV_DEVINL double power(double v, const float2* tab) {
  const float hi = (float)v;
  return ff_to_double(exp_ff(hi, (float)(v - (double)hi), tab));
}

template <int DT>
SV_DEVINL float load_one(const void* row, long long i) {
  return DT == SV_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(row)[i])
                       : static_cast<const float*>(row)[i];
}

// Eight elements from e on (e a multiple of 8); -inf from `end` on. VEC: rows
// are 16-byte aligned.
template <int DT, bool VEC>
SV_DEVINL void load8(const void* row, int e, int end, float2 (&v)[4]) {
  if (VEC && e + 8 <= end) {
    if constexpr (DT == SV_BF16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + e);
      v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
      v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
      v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
      v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + e);
      const float4 a = p[0], b = p[1];
      v[0] = make_float2(a.x, a.y);
      v[1] = make_float2(a.z, a.w);
      v[2] = make_float2(b.x, b.y);
      v[3] = make_float2(b.z, b.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i].x = e + 2 * i < end ? load_one<DT>(row, e + 2 * i) : neg_inf();
      v[i].y = e + 2 * i + 1 < end ? load_one<DT>(row, e + 2 * i + 1) : neg_inf();
    }
  }
}

// exp((l - m)/T) of a pair as float-floats, to about 1e-12.
SV_DEVINL ff2 weight2(float2 l, float nm, const Args& a, const float2* tab) {
  const ff2 x = scaled_diff2(l, f2(nm), a.ih, a.il, a.unit_t != 0);
  return exp_ff2(x.hi, x.lo, tab);
}

// A pass's weights: w(x) = e_q max(0, a - b e^d) with e_q = exp((lq - mq)/T) and
// d = ((lp - mp) - (lq - mq))/T, or e_q alone (`plain`). With a = A and
// b = B S_q/S_p this is S_q max(0, A q - B p), q's factor taken out: where A q and
// B p nearly cancel, the error is then that of the ratio p/q alone, and tokens of
// one logit difference keep their exact proportions. d is formed as
// (lp - lq) + (mq - mp) for the same reason.
struct Mix {
  const void *q, *p;
  float nmq;     // -mq
  ff c;          // mq - mp
  ff a, b;
  bool plain;
  // With `shorter` (row maxima and their difference within 1500 T) the weights come from
  // exp_draw2 on the logits as they are, to 5e-11: q's relative to 2^q0 (qb is 127 - q0), the
  // ratio's times 2^n (rb is 127 + n, and b takes the rest of exp((mq - mp)/T)); top is the
  // largest difference whose ratio stays in range.
  bool shorter;
  int qb, rb;
  float top;
};

// Ratios above e^80 count as e^80: their weight is 0 unless b < a e^-80.
constexpr float kRatioTop = 80.0f;

// e_q of a pair of logits of q (or of p, with its own qb).
SV_DEVINL ff2 short2(float2 l, int qb, const Args& a, const float2* tab1k) {
  l = make_float2(fmaxf(l.x, -a.reach), fmaxf(l.y, -a.reach));
  return exp_draw2(l, make_int2(qb, qb), a.dc, tab1k);
}

SV_DEVINL ff2 plain2(float2 l, const Mix& x, const Args& a, const float2* tab, const float2* tab1k) {
  return x.shorter ? short2(l, x.qb, a, tab1k) : weight2(l, x.nmq, a, tab);
}

// a - b r, then times e; 0 where that is not positive.
SV_DEVINL ff2 mixed(const ff2& e, const ff2& r, const Mix& x) {
  const float2 ph = f2_mul(r.hi, f2(-x.b.hi));
  const float2 pe = f2_fma(r.hi, f2(-x.b.hi), f2_mul(ph, f2(-1.0f)));
  const float2 pl = f2_sub(pe, f2_fma(r.hi, f2(x.b.lo), f2_mul(r.lo, f2(x.b.hi))));
  const ff2 t0 = two_sum2(f2(x.a.hi), ph);
  // (Normalised: where the heads cancel, the tails are all there is.)
  const ff2 t = two_sum2(t0.hi, f2_add(t0.lo, f2_add(f2(x.a.lo), pl)));
  const float2 wh = f2_mul(e.hi, t.hi);
  const float2 we = f2_fma(e.hi, t.hi, f2_mul(wh, f2(-1.0f)));
  const float2 wl = f2_add(we, f2_fma(e.hi, t.lo, f2_mul(e.lo, t.hi)));
  const bool kx = e.hi.x > 0.0f && t.hi.x > 0.0f, ky = e.hi.y > 0.0f && t.hi.y > 0.0f;
  return {make_float2(kx ? wh.x : 0.0f, ky ? wh.y : 0.0f),
          make_float2(kx ? wl.x : 0.0f, ky ? wl.y : 0.0f)};
}

SV_DEVINL ff2 mix2_short(float2 lq, float2 lp, const Mix& x, const Args& a, const float2* tab1k) {
  const ff2 e = short2(lq, x.qb, a, tab1k);
  ff2 d = two_sum2(lp, f2_mul(lq, f2(-1.0f)));
  if (!(d.hi.x < x.top)) d.hi.x = x.top, d.lo.x = 0.0f;  // (also where the target has no such token)
  if (!(d.hi.y < x.top)) d.hi.y = x.top, d.lo.y = 0.0f;
  if (d.hi.x < -a.reach) d.hi.x = -a.reach, d.lo.x = 0.0f;
  if (d.hi.y < -a.reach) d.hi.y = -a.reach, d.lo.y = 0.0f;
  ff2 r = exp_draw2(d.hi, make_int2(x.rb, x.rb), a.dc, tab1k);
  r.lo = f2_fma(r.hi, f2_mul(d.lo, f2(a.ih)), r.lo);
  return mixed(e, r, x);
}

SV_DEVINL ff2 mix2(float2 lq, float2 lp, const Mix& x, const Args& a, const float2* tab) {
  const ff2 e = weight2(lq, x.nmq, a, tab);
  const ff2 d0 = two_sum2(lp, f2_mul(lq, f2(-1.0f)));
  const ff2 d1 = two_sum2(d0.hi, f2(x.c.hi));
  ff2 d = {d1.hi, f2_add(d1.lo, f2_add(d0.lo, f2(x.c.lo)))};
  if (a.unit_t == 0) {
    const float2 h = f2_mul(d.hi, f2(a.ih));
    const float2 r = f2_fma(d.hi, f2(a.ih), f2_mul(h, f2(-1.0f)));
    d.lo = f2_fma(d.hi, f2(a.il), f2_fma(d.lo, f2(a.ih), r));
    d.hi = h;
  }
  if (d.hi.x > kRatioTop) d.hi.x = kRatioTop, d.lo.x = 0.0f;
  if (d.hi.y > kRatioTop) d.hi.y = kRatioTop, d.lo.y = 0.0f;
  const ff2 r = exp_ff2(d.hi, d.lo, tab);
  return mixed(e, r, x);
}

template <int DT, bool VEC>
SV_DEVINL void mix8(const Mix& x, int e, int end, const Args& a, const float2* tab, const float2* tab1k,
                    ff2 (&w)[4]) {
  float2 q[4];
  load8<DT, VEC>(x.q, e, end, q);
  if (x.plain) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = plain2(q[i], x, a, tab, tab1k);
    return;
  }
  float2 p[4];
  load8<DT, VEC>(x.p, e, end, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = x.shorter ? mix2_short(q[i], p[i], x, a, tab1k) : mix2(q[i], p[i], x, a, tab);
}

// fp64 runs at a 64th of the fp32 rate here: it is left to one warp's decisions, and
// sums are float-floats (about 2^-44).
SV_DEVINL ff ff2_warp_sum(const ff2& s) {
  return ff_warp_sum(ff_add({s.hi.x, s.lo.x}, {s.hi.y, s.lo.y}));
}

// Maximum and sum of exp((l - max)/T), in fp32, over a warp's region of one or two
// rows, in one pass: a lane's running maximum moves at most once for eight elements.
// NaN and +inf end in a NaN sum; a region of -inf has the maximum -inf and the sum 0.
struct Running {
  float m, s;
  SV_DEVINL void take(const float2 (&v)[4], float c2) {
    float top = m;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(v[i].x, v[i].y));
    const float ref = top == neg_inf() ? 0.0f : top;
    float2 acc[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = f2_mul(f2_add(v[i], f2(-ref)), f2(c2));
      acc[i & 1] = f2_add(acc[i & 1], make_float2(ex2_fast(y.x), ex2_fast(y.y)));
    }
    const float2 t = f2_add(acc[0], acc[1]);
    const float keep = top > m ? ex2_fast((m - ref) * c2) : 1.0f;  // m = -inf: 0 (and s = 0)
    s = fmaf(s, keep, t.x + t.y);
    m = top;
  }
  SV_DEVINL void over_warp(float c2) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      const float top = fmaxf(m, m2);
      const float ref = top == neg_inf() ? 0.0f : top;
      s = (m == neg_inf() ? s : s * ex2_fast((m - ref) * c2)) + (m2 == neg_inf() ? s2 : s2 * ex2_fast((m2 - ref) * c2));
      m = top;
    }
  }
};

template <int DT, bool VEC>
SV_DEVINL void region_stats(const void* q, const void* p, int begin, int end, int lane, const Args& a, Running (&r)[2]) {
  r[0] = r[1] = {neg_inf(), 0.0f};
  if (p) {
#pragma unroll 2
    for (int e = begin + lane * 8; e < end; e += kStep) {
      float2 v[4], w[4];
      load8<DT, VEC>(q, e, end, v);
      load8<DT, VEC>(p, e, end, w);
      r[0].take(v, a.c2);
      r[1].take(w, a.c2);
    }
    r[1].over_warp(a.c2);
  } else {
#pragma unroll 2
    for (int e = begin + lane * 8; e < end; e += kStep) {
      float2 v[4];
      load8<DT, VEC>(q, e, end, v);
      r[0].take(v, a.c2);
    }
  }
  r[0].over_warp(a.c2);
}

// The same sum as a float-float, of a row's weights as the draw takes them.
template <int DT, bool VEC>
SV_DEVINL ff region_sum(const Mix& x, int begin, int end, int lane, const Args& a, const float2* tab,
                        const float2* tab1k) {
  ff2 acc = {f2(1.0f), f2(0.0f)};
#pragma unroll 1
  for (int e = begin + lane * 8; e < end; e += kStep) {
    float2 v[4];
    load8<DT, VEC>(x.q, e, end, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) ff_accumulate_biased2(acc, plain2(v[i], x, a, tab, tab1k));
  }
  acc.hi = f2_add(acc.hi, f2(-1.0f));
  return ff2_warp_sum(acc);
}

// Sum of the residual's weights over a warp's region.
template <int DT, bool VEC>
SV_DEVINL ff region_mix(const Mix& x, int begin, int end, int lane, const Args& a, const float2* tab,
                        const float2* tab1k) {
  ff2 acc = {f2(0.0f), f2(0.0f)};
#pragma unroll 1
  for (int e = begin + lane * 8; e < end; e += kStep) {
    ff2 w[4];
    mix8<DT, VEC>(x, e, end, a, tab, tab1k, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ff2 s = two_sum2(acc.hi, w[i].hi);
      acc.hi = s.hi;
      acc.lo = f2_add(acc.lo, f2_add(s.lo, w[i].lo));
    }
  }
  return ff2_warp_sum(acc);
}

// exp(((lq - mq) - (lp - mp))/T), c = mq - mp: from the difference of the logits, so
// that it holds where both probabilities are too small for fp32. Beyond e^80 it
// is infinite, below e^-87 a positive 1e-40; 0 where the target has no such token.
SV_DEVINL double token_ratio(float lq, float lp, ff c, const Args& a, const float2* tab) {
  if (lq == neg_inf()) return 0.0;
  if (lp == neg_inf()) return INFINITY;
  const ff d0 = two_sum(lq, -lp);
  const ff d1 = two_sum(d0.hi, -c.hi);
  const float dl = __fadd_rn(d1.lo, __fsub_rn(d0.lo, c.lo));
  const ff h = two_prod(d1.hi, a.ih);
  const float hl = __fmaf_rn(d1.hi, a.il, __fmaf_rn(dl, a.ih, h.lo));
  if (h.hi > kRatioTop) return INFINITY;
  if (h.hi < -87.0f) return 1e-40;
  return ff_to_double(exp_ff(h.hi, hl, tab));
}

// The token at which the running sum of the region's weights passes `target`,
// or the region's last token of positive weight. The lanes' running sums are of
// one order each, so that rounding alone may lift a lane without weight over a target at
// the border before it: then the token before the border is drawn, the one after where
// the region has none before.
template <int DT, bool VEC>
SV_DEVINL int region_draw(const Mix& x, int begin, int end, ff target, int lane, const Args& a,
                          const float2* tab, const float2* tab1k) {
  ff before = {0.0f, 0.0f};
  int last = -1;
#pragma unroll 1
  for (int e0 = begin; e0 < end; e0 += kStep) {
    const int e = e0 + lane * 8;
    const int earlier = last;
    ff2 w[4];
    mix8<DT, VEC>(x, e, end, a, tab, tab1k, w);
    ff mine = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mine = ff_add(mine, {w[i].hi.x, w[i].lo.x});
      mine = ff_add(mine, {w[i].hi.y, w[i].lo.y});
      if (w[i].hi.x > 0.0f) last = e + 2 * i;
      if (w[i].hi.y > 0.0f) last = e + 2 * i + 1;
    }
    ff incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const ff t = ff_shfl_up(incl, o);
      if (lane >= o) incl = ff_add(incl, t);
    }
    const unsigned hit = __ballot_sync(0xffffffffu, ff_gt(ff_add(before, incl), target));
    if (hit) {
      const int owner = __ffs(hit) - 1;
      int token = -1, first = INT_MAX;
      ff run = ff_add(before, ff_sub(incl, mine));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const ff v = i & 1 ? ff{w[i >> 1].hi.y, w[i >> 1].lo.y} : ff{w[i >> 1].hi.x, w[i >> 1].lo.x};
        run = ff_add(run, v);
        if (v.hi > 0.0f) first = min(first, e + i);
        if (token < 0 && v.hi > 0.0f && ff_gt(run, target)) token = e + i;
      }
      token = __shfl_sync(0xffffffffu, token, owner);
      if (token >= 0) return token;
      token = __reduce_max_sync(0xffffffffu, lane <= owner ? last : earlier);
      if (token >= 0) return token;
      first = __reduce_min_sync(0xffffffffu, lane > owner ? first : INT_MAX);
      if (first < INT_MAX) return first;
    }
    before = ff_add(before, {__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)});
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
  return last;
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) tree_verify_kernel(Args a, int nc) {
  __shared__ Shared sh;
  constexpr int kEs = DT == SV_BF16 ? 2 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = cluster_ctarank();
  const long long b = blockIdx.x / nc;
  const int T = a.T;
  sh.tab[tid] = kSvExp2Table[tid];
#pragma unroll
  for (int i = 0; i < 1024; i += kThreads) sh.tab1k[tid + i] = kSvExp2Table1024[tid + i];

  // ---- the tree, checked by every CTA alike
  unsigned bad = 0;
  if (tid < T) {
    const long long at = b * T + tid;
    const int p = a.parents[at];
    sh.parents[tid] = p;
    sh.tokens[tid] = a.tokens[at];
    sh.u[tid] = a.uniforms[at];
    sh.drow[tid] = a.draft_index[at];
  }
  __syncthreads();
  if (tid < T) {
    const int p = sh.parents[tid];
    if (tid == 0 ? p != -1 : (p != -2 && (p < 0 || p >= tid || sh.parents[p] == -2))) bad |= SV_DEV_TREE;
    if (p != -2) {
      if (!(sh.u[tid] >= 0.0f && sh.u[tid] <= 1.0f)) bad |= SV_DEV_UNIFORM_RANGE;
      if (tid > 0 && (sh.tokens[tid] < 0 || sh.tokens[tid] >= a.V)) bad |= SV_DEV_TOKEN_RANGE;
      if (tid > 0 && p >= 0 && p < tid && (sh.drow[p] < 0 || sh.drow[p] >= a.R)) bad |= SV_DEV_TREE;
    }
  }
  if (bad && rank == 0) atomicOr(a.status, bad);
  const bool failed_args = __syncthreads_or(bad != 0);
  int32_t* out = a.out_tokens + b * T;
  int32_t* nodes = a.out_nodes + b * T;
  if (failed_args) {  // every CTA of the cluster comes here
    if (rank == 0) {
      for (int i = tid; i < T; i += kThreads) out[i] = nodes[i] = -1;
      if (tid == 0) a.n_acc[b] = -1;
    }
    return;
  }
  cluster_sync();  // every CTA has started: its shared memory may be written

  const int region0 = (int)(rank * kWarps + warp);
  const int begin = (int)min((long long)a.V, (long long)region0 * a.region);
  const int end = (int)min((long long)a.V, (long long)begin + a.region);
  unsigned phase = 0;
  int cur = 0, count = 0, buf = 0;
  unsigned failure = 0;
  Mix x{};
  for (;;) {  // one round a visited node
    bool kids = false;
    for (int i = cur + 1 + tid; i < T; i += kThreads) kids |= sh.parents[i] == cur;
    kids = __syncthreads_or(kids);
    const void* q = static_cast<const unsigned char*>(a.target) + ((b * T + cur) * a.V) * kEs;
    const void* p = kids ? static_cast<const unsigned char*>(a.draft) + (long long)sh.drow[cur] * a.V * kEs
                         : nullptr;
    // ---- maxima and sums of the node's rows
    buf = 0;
    {
      Running r[2];
      region_stats<DT, VEC>(q, p, begin, end, lane, a, r);
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          sh.wtop[k][warp] = r[k].m;
          sh.wfast[k][warp] = r[k].s;
        }
      }
    }
    __syncthreads();
    Exchange& ex = sh.x[phase & 1];
    ++phase;
    // Warp 0 joins q's regions, warp 1 p's. (A region's sum may be NaN although
    // its maximum is -inf: it counts.)
    auto joined = [&](float t, float own, float* m) {
      float top = t;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      *m = top;
      float sum = own == 0.0f ? 0.0f : t == neg_inf() ? own : own * ex2_fast((t - top) * a.c2);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      return sum;
    };
    if (warp < (kids ? 2 : 1)) {
      const int r = warp;
      float m;
      const float sum = joined(lane < kWarps ? sh.wtop[r][lane] : neg_inf(), lane < kWarps ? sh.wfast[r][lane] : 0.0f, &m);
      if (lane < nc) {
        dsmem_st_f32x2(dsmem_map(smem_u32(&ex.sum[r][rank]), lane), sum, 0.0f);
        dsmem_st_f32(dsmem_map(smem_u32(&ex.top[r][rank]), lane), m);
      }
    }
    cluster_sync();
    if (warp < (kids ? 2 : 1)) {
      const int r = warp;
      float m;
      const float sum = joined(lane < nc ? ex.top[r][lane] : neg_inf(), lane < nc ? ex.sum[r][lane].hi : 0.0f, &m);
      if (lane == 0) {
        sh.m[r] = m;
        sh.S[r] = (double)sum;
      }
    }
    __syncthreads();
    x = Mix{};
    x.q = q;
    x.p = p;
    x.nmq = -sh.m[0];
    x.plain = true;
    if (kids) x.c = two_sum(sh.m[0], -sh.m[1]);
    const float mq = sh.m[0], mp = kids ? sh.m[1] : sh.m[0];
    const float near = 0.75f * a.reach;
    x.shorter = a.short_ok && fabsf(mq) < near && fabsf(mp) < near && fabsf(mq - mp) < near;
    Mix xp = x;  // the draft row alone
    xp.q = p;
    xp.nmq = -mp;
    int n2 = 0;
    if (x.shorter) {
      const int q0 = (int)floorf(mq * a.c2) + 1, p0 = (int)floorf(mp * a.c2) + 1;
      n2 = (int)rintf((mq - mp) * a.c2);
      x.qb = 127 - q0;
      xp.qb = 127 - p0;
      x.rb = 127 + n2;
      x.top = fminf(a.reach, (float)(126 - n2) / a.c2);
    }

    // ---- the children in turn, by warp 0 of each CTA alike; the others serve its passes
    double A = 1.0, Bp = 0.0, scale = 1.0, p_over_q = 1.0, Sq = 1.0;
    int i = cur + 1;
    if (warp == 0) {
      unsigned f = 0;
      for (int r = 0; r < (kids ? 2 : 1); ++r) {
        if (!(sh.S[r] < INFINITY) || sh.m[r] == INFINITY) f |= SV_DEV_NONFINITE;
        else if (sh.m[r] == neg_inf()) f |= SV_DEV_EMPTY_ROW;
      }
      if (lane == 0) sh.failure = f;
      if (kids && !f) {
        p_over_q = sh.S[1] / sh.S[0];
        for (int k = cur + 1 + lane; k < T; k += 32)
          if (sh.parents[k] == cur)
            sh.ratio[k] = token_ratio(load_one<DT>(q, sh.tokens[k]), load_one<DT>(p, sh.tokens[k]), x.c, a, sh.tab);
      }
      __syncwarp();
    }
    int next;
    bool precise = false;  // the sums in float-floats are at hand
    for (;;) {
      if (warp == 0) {
        int to = kDraw;
        for (; i < T; ++i) {
          if (sh.parents[i] != cur) continue;
          // r(x)/p(x) = A q/p - B
          to = (double)sh.u[i] < fmin(1.0, A * (sh.ratio[i] * p_over_q) - Bp) ? i : kResidual;
          ++i;
          break;
        }
        if (lane == 0) sh.next = to;
      }
      __syncthreads();
      next = sh.next;
      failure = sh.failure;
      if (failure || next >= 0) break;
      if (!precise) {
        precise = true;
        const int rows = next == kResidual ? 2 : 1;
#pragma unroll 1
        for (int r = 0; r < rows; ++r) {
          const ff sum = region_sum<DT, VEC>(r ? xp : x, begin, end, lane, a, sh.tab, sh.tab1k);
          if (lane == 0) sh.wsum[0][r][warp] = sum;
        }
        __syncthreads();
        Exchange& ep = sh.x[phase & 1];
        ++phase;
        if (warp < rows) {
          const ff c = ff_warp_sum(lane < kWarps ? sh.wsum[0][warp][lane] : ff{0.0f, 0.0f});
          if (lane < nc) dsmem_st_f32x2(dsmem_map(smem_u32(&ep.sum[warp][rank]), lane), c.hi, c.lo);
        }
        cluster_sync();
        if (warp == 0) {
          const ff c = lane < nc ? ep.sum[0][lane] : ff{0.0f, 0.0f};
          if (lane < nc) sh.cta_sum[0][lane] = c;
          Sq = ff_to_double(ff_warp_sum(c));
          if (rows == 2) {
            p_over_q = ff_to_double(ff_warp_sum(lane < nc ? ep.sum[1][lane] : ff{0.0f, 0.0f})) / Sq;
            // (The short weights' sums are relative to powers of two, not to the maxima.)
            if (x.shorter)
              p_over_q *= power((double)(x.qb - xp.qb) * kLn2 + ((double)mq - (double)mp) * a.inv_t, sh.tab);
          }
        }
        __syncthreads();
      }
      if (next == kDraw) break;
      if (warp == 0) {
        // Scaled by a power of two so that the larger scalar lies in [1, 2).
        const int ex2 = ilogb(fmax(A, Bp + 1.0));
        scale = ldexp(1.0, -ex2);
        const double fa = A * scale;
        double fb = (Bp + 1.0) * scale / p_over_q;
        if (x.shorter) fb *= power(((double)mq - (double)mp) * a.inv_t - (double)n2 * kLn2, sh.tab);
        if (lane == 0) {
          sh.a = {(float)fa, (float)(fa - (double)(float)fa)};
          sh.b = {(float)fb, (float)(fb - (double)(float)fb)};
        }
      }
      __syncthreads();
      Mix y = x;
      y.plain = false;
      y.a = sh.a;
      y.b = sh.b;
      const int nb = buf ^ 1;
      const ff sum = region_mix<DT, VEC>(y, begin, end, lane, a, sh.tab, sh.tab1k);
      if (lane == 0) sh.wsum[nb][0][warp] = sum;
      __syncthreads();
      Exchange& ez = sh.x[phase & 1];
      ++phase;
      if (warp == 0) {
        const ff c = ff_warp_sum(lane < kWarps ? sh.wsum[nb][0][lane] : ff{0.0f, 0.0f});
        if (lane < nc) dsmem_st_f32x2(dsmem_map(smem_u32(&ez.sum[0][rank]), lane), c.hi, c.lo);
      }
      cluster_sync();
      if (warp == 0) {
        const ff c = lane < nc ? ez.sum[0][lane] : ff{0.0f, 0.0f};
        if (lane < nc) sh.cta_sum[nb][lane] = c;
        const double Z = ff_to_double(ff_warp_sum(c)) / (Sq * scale);
        const bool keep = Z >= kResidualMin;
        if (keep) {
          const double inv = 1.0 / Z;
          A *= inv;
          Bp = (Bp + 1.0) * inv;
        }
        if (lane == 0) sh.keep = keep;
      }
      __syncthreads();
      if (sh.keep) {
        x = y;
        buf = nb;
      }
    }
    __syncthreads();  // sh.next and sh.failure have been read
    if (failure || next < 0) break;
    if (tid == 0) sh.path[count] = next;
    ++count;
    cur = next;
  }

  if (failure) {
    if (rank == 0) {
      if (tid == 0) {
        atomicOr(a.status, failure);
        a.n_acc[b] = -1;
      }
      for (int i = tid; i < T; i += kThreads) out[i] = nodes[i] = -1;
    }
    return;
  }

  // ---- the draw: the CTA, then the warp whose region holds u * total
  if (rank == 0) {
    for (int i = tid; i < T; i += kThreads) {
      const int node = i < count ? sh.path[i] : -1;
      nodes[i] = node;
      if (i != count) out[i] = node < 0 ? -1 : sh.tokens[node];
    }
    if (tid == 0) a.n_acc[b] = count;
  }
  ff total = {0.0f, 0.0f};
  for (int c = 0; c < nc; ++c) total = ff_add(total, sh.cta_sum[buf][c]);
  const ff goal = ff_mul_f(total, sh.u[0]);
  ff before = {0.0f, 0.0f}, at = {0.0f, 0.0f};
  int owner = -1, last = 0;
  for (int c = 0; c < nc; ++c) {
    const ff s = sh.cta_sum[buf][c];
    const ff upto = ff_add(before, s);
    if (s.hi > 0.0f) {
      last = c;
      if (owner < 0 && ff_gt(upto, goal)) {
        owner = c;
        at = before;
      }
    }
    before = upto;
  }
  const bool past = owner < 0;  // u = 1: the last token of positive weight
  if (past) owner = last;
  if (owner != (int)rank) return;
  before = at;
  int w = -1;
  last = 0;
  for (int i = 0; i < kWarps; ++i) {
    const ff s = sh.wsum[buf][0][i];
    const ff upto = ff_add(before, s);
    if (s.hi > 0.0f) {
      last = i;
      if (w < 0 && !past && ff_gt(upto, goal)) {
        w = i;
        at = before;
      }
    }
    before = upto;
  }
  const bool beyond = w < 0;
  if (beyond) w = last;
  if (w != warp) return;
  const ff rest = beyond ? ff{INFINITY, 0.0f} : ff_sub(goal, at);
  const int token = region_draw<DT, VEC>(x, begin, end, rest, lane, a, sh.tab, sh.tab1k);
  if (lane == 0) out[count] = token;
}

// ---------------------------------------------------------------- host side

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

bool sizes_ok(int B, int T, int V, int dtype) {
  if (dtype != SV_BF16 && dtype != SV_F32) return false;
  if (B < 0 || T < 1 || T > kTreeMax || V < 1 || V > (1 << 30)) return false;
  return (long long)B * T * V <= (1ll << 45) && B <= (1 << 27);
}

// CTAs a sequence: each warp gets a step of 256 elements at least, up to the
// portable cluster size.
int cluster_size(int V) {
  int nc = 1;
  while (nc < kMaxCluster && (long long)nc * kWarps * kStep < V) nc <<= 1;
  return nc;
}

template <int DT, bool VEC>
cudaError_t launch(const Args& a, cudaStream_t st) {
  const int nc = cluster_size(a.V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B * (unsigned)nc);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<DT, VEC>, a, nc);
}

}  // namespace tvf
}  // namespace sv

using namespace sv::tvf;

extern "C" {

size_t sv_tree_workspace_size(int B, int T, int V, int dtype) {
  return sizes_ok(B, T, V, dtype) ? 256 : 0;
}

int spec_verify_tree(const void* target_logits, const void* draft_logits, const int32_t* draft_index,
                     const int32_t* tokens, const int32_t* parents, const float* uniforms, int B, int T,
                     int V, int R, int dtype, float temperature, int32_t* out_tokens,
                     int32_t* out_nodes, int32_t* n_accepted, void* workspace, size_t workspace_bytes,
                     void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  if (!sizes_ok(B, T, V, dtype) || R < 0) return SV_ERR_SHAPE;
  if (!std::isfinite(temperature) || !(temperature > 0.0f)) return SV_ERR_TEMPERATURE;
  if (B == 0) return SV_OK;
  if (!target_logits || (R > 0 && !draft_logits) || !draft_index || !tokens || !parents || !uniforms ||
      !out_tokens || !out_nodes || !n_accepted || !workspace)
    return SV_ERR_NULL;
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (misaligned(target_logits, es) || misaligned(draft_logits, es) || misaligned(draft_index, 4) ||
      misaligned(tokens, 4) || misaligned(parents, 4) || misaligned(uniforms, 4) ||
      misaligned(out_tokens, 4) || misaligned(out_nodes, 4) || misaligned(n_accepted, 4) ||
      misaligned(workspace, 256))
    return SV_ERR_ALIGN;
  if (workspace_bytes < sv_tree_workspace_size(B, T, V, dtype)) return SV_ERR_WORKSPACE;
  Args a{};
  a.target = target_logits;
  a.draft = draft_logits;
  a.draft_index = draft_index;
  a.tokens = tokens;
  a.parents = parents;
  a.uniforms = uniforms;
  a.out_tokens = out_tokens;
  a.out_nodes = out_nodes;
  a.n_acc = n_accepted;
  a.status = static_cast<unsigned*>(workspace);
  a.B = B;
  a.T = T;
  a.V = V;
  a.R = R;
  const long long regions = (long long)cluster_size(V) * kWarps;
  a.region = (int)(((V + regions - 1) / regions + 7) / 8 * 8);
  const double inv = 1.0 / (double)temperature;
  a.ih = (float)inv;
  a.il = (float)(inv - (double)a.ih);
  a.unit_t = temperature == 1.0f;
  a.c2 = (float)(1.4426950408889634074 * inv);
  a.inv_t = inv;
  {
    const double C = (double)temperature * 0.69314718055994530942 / 1024.0;
    a.dc.ch = (float)C;
    a.dc.cli = (float)((C - (double)a.dc.ch) * inv);
    a.dc.inv = (float)(1.0 / C);
    a.dc.ih = a.ih;
  }
  a.reach = 2000.0f * temperature;
  a.short_ok = temperature >= 1e-3f && temperature <= 1e3f;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SV_ERR_CUDA;
  const bool vec = !misaligned(target_logits, 16) && !misaligned(draft_logits, 16) && (size_t)V * es % 16 == 0;
  cudaError_t e;
  if (dtype == SV_BF16)
    e = vec ? launch<SV_BF16, true>(a, st) : launch<SV_BF16, false>(a, st);
  else
    e = vec ? launch<SV_F32, true>(a, st) : launch<SV_F32, false>(a, st);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
