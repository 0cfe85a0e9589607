// Sampling with temperature, top-k, top-p and min-p from given uniforms
// (spec_filtered_sample): one token a row, from the softmax of the entries that a row's
// own settings keep.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace fs {

typedef unsigned long long u64;

// The kept entries are a prefix of the row in the order of logits, so that a row needs its
// cut, the last entry that is kept. A cluster of CTAs shares a row and passes over it twice, the first time
// from memory and then, as a rule, from L2:
//   1. the maximum, for top_p the sum of all weights in fp32, and counts of a sample of the tiles' entries by
//      value; from them a window of values that the cut is expected in, a few standard deviations of the sample wide;
//   2. the entries of the window and above go to lists in shared memory, to be taken by full
//      warps: those above are weighed and summed, those within are set aside and counted into the bins of a histogram,
//      by number and mass. The entries of the cut's bin go to every CTA, which puts them in order; the
//      kept ones' weights join the sums;
//   3. the sums are kept by ranges of ids (records: what a warp has summed up between two turns of its
//      list), so that the uniform's range is known, and its token is found there.
// The CTAs wait for one another once after each of these steps, and once for the cut's bin. All decisions are made on
// whole-number masses (2^-44 of the largest weight), where sums do not depend on their order. Where the fp32
// sum could change the cut, the mass below the window is summed again, exactly. A window that misses the cut
// is widened, or begins above its old top where the cut turns out to lie there; one with more entries than there is room for
// (flat rows) is followed by one of three of its bins. A row that still has none, whose cut lies among more
// than a thousand equal entries, or whose top_k is larger than that room and followed by top_p, is halved bit by bit over
// the keys, a pass for every bit.
//
// Few rows are bound by the steps between the passes, each a chain of shared memory, barriers and code fetched for the
// first time (1 x 32000 with top-k: 20 us, of them 8 for the passes). Many rows fill neither issue slots (58 % of them for the
// nucleus rows, 80 to 94 % on the busiest SM) nor memory: a warp's time goes to results of its own instructions (21 %), loads (16 %),
// barriers (11 %) and fetching code (9 %). 512 x 128256 bf16 of normal logits (sigma 3, T = 1), 131 MB, 19 us at the copy
// rate: min_p 0.1 66 us, greedy 76, top_k 50 98, no setting 132 (every entry weighed to 2^-44), top_p 0.9 197, and 626 at T =
// 10, where the window is narrowed. A search bit by bit takes 33 passes: 64 x 128256 bf16 with top_k 60000 and top_p 1165.
// A row is shared by as many CTAs as one wave of four an SM holds, then by one for 65536 entries (32768 of fp32):
// with twice as many 512 rows took 234 us against 224 and, with top-k, 126 against 109: what a CTA does between the
// passes is the larger part.

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 256;        // elements of a warp's step: 8 a lane
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;        // bins of the window
constexpr int kSampleBins = 512;  // bins of the sample below the maximum
constexpr int kValueBins = 1024;  // bins by value, over and over again
constexpr int kList = 288;        // listed entries of a warp: a tile's, and fewer than 32 left over
constexpr int kAsideBytes = 14336; // entries of a CTA set aside: 3584 short or 1792 long ones
constexpr int kShortIds = 65536;  // ids of a CTA's share that a short entry can tell apart
constexpr int kCand = 1024;       // entries of the cut's bin
constexpr int kRecords = 64;      // ranges of ids of a warp

struct Args {
  const void* logits;
  long long stride;
  const float* uniforms;
  const float *temp, *top_p, *min_p;
  const int32_t* top_k;
  float temp1, top_p1, min_p1;
  int top_k1;
  int N, V, nc, share, step, scale_bits;
  int32_t* out;
  float* prob;
  unsigned* status;
};

// What a row's weights are made of: w(l) = exp((l - m)/T) times a power of two, as a whole number of
// 2^-scale_bits. The exponential takes l `unit` + `off` as its argument, whose temperature T `unit` lies in [1, 4) (below only
// where T is subnormal). off is 0 where |m/T| < 1386. Elsewhere it is -m unit: the entries that then weigh anything lie
// within 88 T of m, hence within a factor of two of it, and l - m is exact.
struct Weigh {
  int shift;  // of a weight's 45 bits at k >> 10 = 0
  DrawConst dc;
  float unit, off, lmin;
};

// A listed entry: value and place in the CTA's share; a bf16 value and 16 bits of place where those do.
template <bool SHORT>
struct Entry {
  typedef u64 Word;
  static SV_DEVINL u64 make(uint32_t value, int at) { return (u64)value << 32 | (unsigned)at; }
  static SV_DEVINL float value(u64 w) { return __uint_as_float((unsigned)(w >> 32)); }
  static SV_DEVINL int at(u64 w) { return (int)(unsigned)w; }
};
template <>
struct Entry<true> {
  typedef uint32_t Word;
  static SV_DEVINL uint32_t make(uint32_t value, int at) { return value | (unsigned)at; }  // (value: the high half)
  static SV_DEVINL float value(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  static SV_DEVINL int at(uint32_t w) { return (int)(w & 0xffffu); }
};

struct Shared {
  float2 tab[1024];
  union {
    u64 list[kWarps][kList];  // of either kind of entry
    u64 cand[kCand];          // key, then ~id: entries of the cut's bin
  };
  union {
    u64 aside[kAsideBytes / 8];  // of either kind
    unsigned sample[kValueBins];
  };
  unsigned hlo[kBins], hhi[kBins], hcnt[kBins];
  unsigned rec_lo[kWarps][kRecords], rec_hi[kWarps][kRecords];
  int rec_end[kWarps][kRecords];  // the id behind the record's last one
  int recs[kWarps];
  u64 wsum[2][kWarps];
  unsigned wcnt[2][kWarps], wmore[2][kWarps];
  u64 bins_sum[kWarps];  // the window's bins, a warp's
  unsigned bins_cnt[kWarps];
  u64 inbox[2][kMaxCluster];
  unsigned inbox_c[2][kMaxCluster], inbox_d[2][kMaxCluster];
  u64 tile_sum[kWarps], hit_start;
  int hit_from, hit_to;
  float fmass[kWarps], fvar[kWarps], wmax[kWarps];
  u64 cta_sum[kMaxCluster];
  float cta_max[kMaxCluster];
  unsigned cta_sampled[kMaxCluster];
  unsigned n_aside, n_cand[4];
  int edge[2], bin;  // edges: the window's upper and lower one
  // What the last attempt says of the cut: it lies at or above next_lo, and not above next_hi.
  bool given;
  float next_lo, next_hi;
  u64 bin_mass;
  unsigned bin_count;
  // The cut: entries of a larger key are kept, and those of this key up to `cut_id`; their mass.
  unsigned cut_key;
  int cut_id, cut_found;
  u64 cut_mass;
  float log_hi, log_lo;  // T ln(min_p), times the weights' unit
  Weigh w;
};

SV_DEVINL float unordered(unsigned k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
// The next value above x.
SV_DEVINL float just_above(float x) {
  return x == 0.0f ? __uint_as_float(1u) : __uint_as_float(__float_as_uint(x) + (x > 0.0f ? 1u : 0xffffffffu));
}
// The largest value that compares below x: for -FLT_MAX -inf, and for zeros (of either sign) the first below both.
SV_DEVINL float just_below(float x) { return unordered(min(ordered(x) - 1u, x == 0.0f ? 0x7ffffffeu : 0xffffffffu)); }

// The weight of l (-inf: 0).
SV_DEVINL u64 weight(float l, const Weigh& w, const float2* tab) {
  // exp_draw's steps up to head + tail = T.x + lo in [1, 2) times 2^(k >> 10), then in whole numbers: the
  // head's 24 bits and the tail's to 2^-40, twice 2^44 of them, shifted into place and rounded.
  const float x = fmaxf(__fmaf_rn(l, w.unit, w.off), w.lmin);
  const float ym = __fmaf_rn(x, -w.dc.inv, kRoundMagic), nkf = __fsub_rn(ym, kRoundMagic);
  const float sv = __fmaf_rn(__fmaf_rn(nkf, w.dc.ch, x), w.dc.ih, __fmul_rn(nkf, w.dc.cli));
  const float u = __fmaf_rn(sv, __fmul_rn(__fmaf_rn(sv, 1.0f / 6.0f, 0.5f), sv), sv);
  const int k = __float_as_int(kRoundMagic) - __float_as_int(ym);
  const float2 T = tab[k & 1023];
  const int tail = __float2int_rn(__fmaf_rn(T.x, u, T.y) * 0x1p40f);  // below 2^31
  const unsigned head = (__float_as_uint(T.x) & 0x7fffffu) | 0x800000u;
  const u64 both = (u64)head * (1u << 22) + (u64)((long long)tail * 32);
  return ((both >> min(w.shift - (k >> 10), 63)) + 1) >> 1;
}

// Eight elements a lane of the tile at `base` of a row, as they are stored (bf16 pairs in the first
// four words, or fp32); -inf beyond `end`. Which id is where: tile_id.
template <bool F32, bool VEC>
SV_DEVINL void load_tile(const void* row, int base, int end, int lane, uint32_t (&w)[F32 ? 8 : 4]) {
  if constexpr (!F32) {
    const int at = base + lane * 8;
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(row) + at;
    if (VEC && at + 8 <= end) {
      const uint4 x = ld_global_nc_v4(p);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned a = at + 2 * i < end ? __bfloat16_as_ushort(p[2 * i]) : 0xff80u;
        const unsigned b = at + 2 * i + 1 < end ? __bfloat16_as_ushort(p[2 * i + 1]) : 0xff80u;
        w[i] = a | b << 16;
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int at = base + q * 128 + lane * 4;
      const float* p = static_cast<const float*>(row) + at;
      if (VEC && at + 4 <= end) {
        const uint4 x = ld_global_nc_v4(p);
        w[4 * q] = x.x, w[4 * q + 1] = x.y, w[4 * q + 2] = x.z, w[4 * q + 3] = x.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * q + i] = __float_as_uint(at + i < end ? p[i] : neg_inf());
      }
    }
  }
}
template <bool F32>
SV_DEVINL int tile_id(int lane, int e) {
  return F32 ? (e >> 2) * 128 + lane * 4 + (e & 3) : lane * 8 + e;
}
template <bool F32>
SV_DEVINL float element(const uint32_t (&w)[F32 ? 8 : 4], int e) {
  if constexpr (F32) return __uint_as_float(w[e]);
  return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
}

SV_DEVINL unsigned dsmem_ld_u32(unsigned a) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
SV_DEVINL u64 dsmem_ld_u64(unsigned a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
SV_DEVINL unsigned dsmem_add_u32(unsigned a, unsigned v) {
  unsigned r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
  return r;
}

// All ones in the halves where a >= b.
SV_DEVINL uint32_t ge2(uint32_t a, uint32_t b) {
  return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
}

// A 64-bit sum in two words of shared memory.
SV_DEVINL void add64(unsigned* lo, unsigned* hi, u64 w) {
  const unsigned l = (unsigned)w, old = atomicAdd(lo, l);
  const unsigned h = (unsigned)(w >> 32) + (old + l < l ? 1u : 0u);
  if (h) atomicAdd(hi, h);
}

SV_DEVINL u64 scan_up(u64 x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
SV_DEVINL unsigned scan_up(unsigned x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Among the n candidates of the cut's bin, the one at which the running count reaches
// `want`, or the running mass does (and does so for every mass from want_lo to want).
// s.bin_mass and s.bin_count are what lies above the bin.
__device__ __noinline__ void order_candidates(Shared& s, int n, bool by_count, u64 want_lo, u64 want) {
  const int tid = threadIdx.x;
  if (tid == 0) s.cut_found = 0;
  u64 mine = 0, x = 0;
  if (n <= kThreads) {
    // A thread a candidate: what stands before it.
    if (tid < n) {
      mine = s.cand[tid];
      x = weight(unordered((unsigned)(mine >> 32)), s.w, s.tab);
      s.cand[kCand / 2 + tid] = x;
    }
    __syncthreads();
    if (tid >= n) return;
    u64 mass = s.bin_mass;
    unsigned count = s.bin_count;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const bool before = s.cand[i] > mine;
      mass += before ? s.cand[kCand / 2 + i] : 0;
      count += before;
    }
    if (by_count ? count + 1 == want : mass < want && mass + x >= want) {
      s.cut_key = (unsigned)(mine >> 32);
      s.cut_id = (int)~(unsigned)mine;
      s.cut_mass = mass + x;
      s.cut_found = by_count || mass < want_lo ? 1 : 2;
    }
    return;
  }
  for (int i = n + tid; i < kCand; i += kThreads) s.cand[i] = 0;
  __syncthreads();
  // Largest first (bitonic).
#pragma unroll 1
  for (int k = 2; k <= kCand; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
#pragma unroll 1
      for (int i = tid; i < kCand / 2; i += kThreads) {
        const int p = 2 * i - (i & (j - 1)), q = p + j;
        const u64 a = s.cand[p], b = s.cand[q];
        if ((p & k) == 0 ? a < b : a > b) s.cand[p] = b, s.cand[q] = a;
      }
      __syncthreads();
    }
  // One warp adds the weights up, 32 at a time.
  if (tid >= 32) return;
  u64 mass = s.bin_mass;
  const unsigned above_count = s.bin_count;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += 32) {
    mine = i0 + tid < n ? s.cand[i0 + tid] : 0;
    x = i0 + tid < n ? weight(unordered((unsigned)(mine >> 32)), s.w, s.tab) : 0;
    const u64 incl = scan_up(x, tid);
    if (i0 + tid < n &&
        (by_count ? above_count + i0 + tid + 1 == want : mass + incl >= want && mass + incl - x < want)) {
      s.cut_key = (unsigned)(mine >> 32);
      s.cut_id = (int)~(unsigned)mine;
      s.cut_mass = mass + incl;
      s.cut_found = by_count || mass + incl - x < want_lo ? 1 : 2;
    }
    mass += __shfl_sync(0xffffffffu, incl, 31);
  }
}

SV_DEVINL float sqrt_fast(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
SV_DEVINL float next_down(float x) { return x * (1.0f - 0x1p-23f); }  // x > 0: below x by one or two steps

// x 2^64, 0 <= x < 1, rounded down.
SV_DEVINL u64 fraction(float x) {
  const unsigned b = __float_as_uint(x);
  const int e = (int)(b >> 23) - 86;  // x = mantissa 2^(e + 86 - 150)
  const u64 mant = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
  return e >= 0 ? mant << e : e > -24 ? mant >> -e : 0;
}

// x 2^e, x >= 0, rounded.
SV_DEVINL u64 whole(float x, int e) {
  const unsigned b = __float_as_uint(x);
  const int sh = (int)(b >> 23) - 150 + e;
  const u64 mant = (b & 0x7fffffu) | 0x800000u;
  return b < 0x800000u || sh < -25 ? 0 : sh >= 0 ? mant << min(sh, 39) : ((mant >> (-sh - 1)) + 1) >> 1;
}

// x / y for 0 < x <= y, to fp32's last place.
SV_DEVINL float ratio(u64 x, u64 y) {
  const float xh = __ull2float_rn(x), yh = __ull2float_rn(y);
  const float xl = __ll2float_rn((long long)(x - __float2ull_rn(xh))), yl = __ll2float_rn((long long)(y - __float2ull_rn(yh)));
  const float q = __fdiv_rn(xh, yh);
  return q + __fdiv_rn(__fmaf_rn(-q, yh, xh) + (xl - q * yl), yh);
}

template <bool F32, bool VEC, bool SHORT>
struct Row {
  static constexpr int WORDS = F32 ? 8 : 4;
  typedef Entry<SHORT> E;
  typedef typename E::Word Word;
  static constexpr unsigned kAside = kAsideBytes / sizeof(Word);
  const Args& a;
  Shared& s;
  const void* row;
  int begin, end, tiles, seg;  // this CTA's ids; tiles in all and of a warp (its segment is contiguous)
  unsigned rank, turn;
  Weigh w;

  SV_DEVINL int lane() const { return threadIdx.x & 31; }
  SV_DEVINL int warp() const { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }
  SV_DEVINL void sync() {
    if (a.nc > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  SV_DEVINL unsigned remote(const void* p, unsigned r) const {
    return a.nc > 1 ? dsmem_map(smem_u32(p), r) : smem_u32(p);
  }
  SV_DEVINL u64 weigh(float l) const { return weight(l, w, s.tab); }

  // Sums over the row's CTAs, the same in every thread. Each CTA's are left in the inboxes of `turn`: another CTA
  // writes them again two sums later, so that the barrier of the sum between says that they have been read.
  // Nothing else may advance `turn`.
  SV_DEVINL void sum(u64& x, unsigned& c, unsigned& d) {
    const int t = turn & 1, ln = lane(), wp = threadIdx.x >> 5;
    ++turn;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    c = __reduce_add_sync(0xffffffffu, c);
    d = __reduce_add_sync(0xffffffffu, d);
    if (ln == 0) s.wsum[t][wp] = x, s.wcnt[t][wp] = c, s.wmore[t][wp] = d;
    __syncthreads();
    if (wp == 0) {
      x = ln < kWarps ? s.wsum[t][ln] : 0;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      x = __shfl_sync(0xffffffffu, x, 0);
      c = __reduce_add_sync(0xffffffffu, ln < kWarps ? s.wcnt[t][ln] : 0u);
      d = __reduce_add_sync(0xffffffffu, ln < kWarps ? s.wmore[t][ln] : 0u);
      if (ln < a.nc) {
        dsmem_st_u64(remote(&s.inbox[t][rank], ln), x);
        dsmem_st_u32(remote(&s.inbox_c[t][rank], ln), c);
        dsmem_st_u32(remote(&s.inbox_d[t][rank], ln), d);
      }
    }
    sync();
    x = 0, c = 0, d = 0;
#pragma unroll 1
    for (int i = 0; i < a.nc; ++i) x += s.inbox[t][i], c += s.inbox_c[t][i], d += s.inbox_d[t][i];
  }
  SV_DEVINL void sum(u64& x, unsigned& c) {
    unsigned d = 0;
    sum(x, c, d);
  }

  // f(first id, words) for tiles first, first + step, ... before `last`, U loaded ahead.
  template <int U, typename F>
  SV_DEVINL void some_tiles(int first, int last, int step, F f) {
#pragma unroll 1
    for (int t0 = first; t0 < last; t0 += U * step) {
      uint32_t x[U][WORDS];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * step;
        load_tile<F32, VEC>(row, begin + t * kTile, t < last ? end : 0, lane(), x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + u * step < last) f(begin + (t0 + u * step) * kTile, x[u]);
    }
  }
  template <int U, typename F>
  SV_DEVINL void all_tiles(F f) {
    some_tiles<U>(warp(), tiles, kWarps, f);
  }

  // Largest element of a lane's eight (no NaN among them).
  SV_DEVINL float top_of(const uint32_t (&x)[WORDS]) {
    if constexpr (F32) {
      float r = __uint_as_float(x[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) r = fmaxf(r, __uint_as_float(x[i]));
      return r;
    } else {
      const uint32_t r = bf16x2_max(bf16x2_max(x[0], x[1]), bf16x2_max(x[2], x[3]));
      return fmaxf(bf16_lo(r), bf16_hi(r));
    }
  }

  SV_DEVINL int bin_of(float l, float top, float per) const {
    return min(kBins - 1, (int)fminf((top - l) * per, (float)kBins));
  }

  // A record of the ids before `stop` that have none yet: the warp's sum of x. A full table is
  // halved first.
  SV_DEVINL void record(int& n, u64 x, int stop) {
    const int ln = lane(), wp = warp();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (n == kRecords) {
      const u64 p = ((u64)s.rec_hi[wp][2 * ln] << 32 | s.rec_lo[wp][2 * ln]) +
                    ((u64)s.rec_hi[wp][2 * ln + 1] << 32 | s.rec_lo[wp][2 * ln + 1]);
      const int e = s.rec_end[wp][2 * ln + 1];
      __syncwarp();
      s.rec_lo[wp][ln] = (unsigned)p, s.rec_hi[wp][ln] = (unsigned)(p >> 32);
      s.rec_end[wp][ln] = e;
      n = kRecords / 2;
      __syncwarp();
    }
    if (ln == 0) {
      s.rec_lo[wp][n] = (unsigned)x, s.rec_hi[wp][n] = (unsigned)(x >> 32);
      s.rec_end[wp][n] = stop;
    }
    ++n;
  }

  // The entries l >= lo of this CTA's share (`all`: every entry): those above hi (and, with a cut, those that it keeps)
  // are summed into records, the others set aside as far as there is room, and all of those counted into bin
  // (top - l) per. Returns a thread's part of the sum.
  SV_DEVINL u64 pass(float lo, float hi, bool cut, bool all, float top, float per, unsigned& count) {
    const int ln = lane(), wp = warp();
    Word* list = reinterpret_cast<Word*>(s.list[wp]);
    Word* aside = reinterpret_cast<Word*>(s.aside);
    const int first = min(tiles, wp * seg), last = min(tiles, first + seg), stop = min(end, begin + last * kTile);
    u64 total = 0;
    int recs = 0;
    count = 0;
    if (all) {
      const int every = (seg + kRecords - 1) / kRecords;
      u64 acc = 0;
      int done = 0;
      some_tiles<2>(first, last, 1, [&](int base, const uint32_t (&x)[WORDS]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc += weigh(element<F32>(x, e));
        if (++done == every) {
          total += acc;
          record(recs, acc, base + kTile);
          acc = 0;
          done = 0;
        }
      });
      total += acc;
      record(recs, acc, stop);
    } else {
      const unsigned key = s.cut_key;
      const int cut_id = s.cut_id;
      int n = 0;
      u64 acc = 0;
      auto take = [&](int from, bool on) {  // 32 entries of the list
        const Word e = list[from + ln];
        const float l = E::value(e);
        bool sure = l > hi;
        if (cut && !sure) {
          const unsigned k = ordered(l);
          sure = k > key || (k == key && begin + E::at(e) <= cut_id);
        }
        const u64 x = on && (sure || !cut) ? weigh(l) : 0;
        if (on && sure) {
          acc += x;
          ++count;
        }
        const bool put = on && !sure && !cut;
        const unsigned b = __ballot_sync(0xffffffffu, put);
        if (b) {
          unsigned at = 0;
          if (ln == 0) at = atomicAdd(&s.n_aside, (unsigned)__popc(b));
          at = __shfl_sync(0xffffffffu, at, 0) + __popc(b & ((1u << ln) - 1));
          if (put) {
            if (at < kAside) aside[at] = e;
            const int bin = bin_of(l, top, per);
            add64(&s.hlo[bin], &s.hhi[bin], x);
            atomicAdd(&s.hcnt[bin], 1u);
          }
        }
      };
      uint32_t lo2 = 0;  // the least bf16 at or above lo, twice
      if constexpr (!F32) {
        const unsigned b = __bfloat16_as_ushort(__float2bfloat16_ru(lo));
        lo2 = b | b << 16;
      }
      // (two tiles of bf16 ahead: 210 us for 512 x 128256 with top-p, 226 with four, whose code is fetched more slowly
      // than it runs, and 216 with one)
      some_tiles<F32 ? 1 : 2>(first, last, 1, [&](int base, const uint32_t (&x)[WORDS]) {
        if (!__any_sync(0xffffffffu, top_of(x) >= lo)) return;
        // In the order of ids: fp32's two halves of a tile one behind the other.
        unsigned mask = 0;
        if constexpr (F32) {
#pragma unroll
          for (int e = 0; e < 8; ++e) mask |= element<F32>(x, e) >= lo ? 1u << e : 0u;
        } else {
          mask = (ge2(x[0], lo2) & 0x00020001u) | (ge2(x[1], lo2) & 0x00080004u) | (ge2(x[2], lo2) & 0x00200010u) |
                 (ge2(x[3], lo2) & 0x00800040u);
          mask = (mask | mask >> 16) & 0xffu;
        }
        const unsigned c = F32 ? __popc(mask & 15u) | __popc(mask >> 4) << 16 : __popc(mask);
        const unsigned incl = scan_up(c, ln), sum = __shfl_sync(0xffffffffu, incl, 31);
        const int head = (int)(sum & 0xffffu), both = head + (int)(sum >> 16);
        if (n + both > kList) {
          __syncwarp();
          const int full = n & ~31;
          for (int i = 0; i < full; i += 32) take(i, true);
          const int stop_at = begin + E::at(list[min(full, kList - 1)]);
          const Word left = list[min(full + ln, kList - 1)];
          total += acc;
          record(recs, acc, full < n ? stop_at : base);
          acc = 0;
          __syncwarp();
          n -= full;
          if (ln < n) list[ln] = left;
        }
        int at = n + (int)((incl - c) & 0xffffu), at2 = n + head + (int)((incl - c) >> 16);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (mask >> e & 1u)
            list[F32 && e >= 4 ? at2++ : at++] = E::make(__float_as_uint(element<F32>(x, e)), base - begin + tile_id<F32>(ln, e));
        n += both;
      });
      __syncwarp();
      for (int i = 0; i < n; i += 32) take(i, i + ln < n);
      total += acc;
      record(recs, acc, stop);
    }
    if (ln == 0) s.recs[wp] = recs;
    return total;
  }

  // The mass of the entries l < lo, exactly (a thread's part).
  SV_DEVINL u64 below(float lo) {
    u64 x = 0;
    all_tiles<1>([&](int, const uint32_t (&v)[WORDS]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float l = element<F32>(v, e);
        const u64 y = weigh(l);
        x += l < lo ? y : 0;
      }
    });
    return x;
  }
};

// The cut of a row by halving: the largest key that the wanted count (K, or 0) or mass reaches, then the last of its
// ties that is kept; into s.cut_key and s.cut_id.
template <bool F32, bool VEC, bool SHORT>
SV_DEVINL void cut_by_bits(Row<F32, VEC, SHORT>& r, unsigned K, bool by_p, u64 part) {
  constexpr int WORDS = F32 ? 8 : 4;
  Shared& s = r.s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto reach = [&](unsigned key, u64& mass, unsigned& count) {  // entries of this key or more
    u64 x = 0;
    unsigned c = 0;
    r.template all_tiles<1>([&](int, const uint32_t (&v)[WORDS]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float l = element<F32>(v, e);
        if (l > neg_inf() && ordered(l) >= key) {
          ++c;
          x += r.weigh(l);
        }
      }
    });
    r.sum(x, c);
    mass = x;
    count = c;
  };
  // Two searches, one after the other, by the same loop: for the count, then for the mass.
  u64 mass = 0, total = 0, want = 0;
  unsigned count = 0, ties = 0xffffffffu, key = 0;
#pragma unroll 1
  for (int by = K ? 0 : 1; by < (by_p ? 2 : 1); ++by) {
    if (by == 1) {
      if (!K) {
        reach(0, mass, count);
        total = mass;
      }
      want = max(__umul64hi(total, part) + (total * part != 0 ? 1u : 0u), (u64)1);
    }
    unsigned found = 0;
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const unsigned tried = found | 1u << bit;
      if (by == 1 && tried <= key) {
        found = tried;  // the k kept entries reach all of their mass
        continue;
      }
      reach(tried, mass, count);
      if (by == 0 ? count >= K : mass >= want) found = tried;
    }
    reach(found + 1, mass, count);
    const u64 one = found ? r.weigh(unordered(found)) : 0;
    if (by == 0) {
      ties = K - count;
      total = mass + ties * one;
    } else {
      const u64 need = one ? (want - mass + one - 1) / one : 1;
      ties = found > key ? (unsigned)need : (unsigned)min((u64)ties, need);
    }
    key = found;
  }
  // The id of the last tie that is kept. A warp's segment is contiguous, and so are the CTAs' shares.
  const int first = min(r.tiles, warp * r.seg), last = min(r.tiles, first + r.seg);
  auto equal = [&](const uint32_t (&v)[WORDS]) {
    unsigned e = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) e += ordered(element<F32>(v, i)) == key;
    return e;
  };
  unsigned mine = 0;
  r.template some_tiles<1>(first, last, 1, [&](int, const uint32_t (&v)[WORDS]) { mine += equal(v); });
  unsigned before = 0, all = mine;
  u64 z = 0;
  const int t = r.turn & 1;
  r.sum(z, all);
  for (int i = 0; i < (int)r.rank; ++i) before += s.inbox_c[t][i];
  for (int i = 0; i < warp; ++i) before += s.wcnt[t][i];
  const unsigned here = s.wcnt[t][warp];
  if (tid == 0) s.cut_id = 0x7fffffff;
  __syncthreads();
  if (all > ties && before < ties && before + here >= ties) {
    unsigned seen = before;
    r.template some_tiles<1>(first, last, 1, [&](int base, const uint32_t (&v)[WORDS]) {
#pragma unroll
      for (int g = 0; g < (F32 ? 2 : 1); ++g) {
        constexpr int PER = F32 ? 4 : 8;
        unsigned e = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) e += ordered(element<F32>(v, g * PER + i)) == key;
        const unsigned inc = scan_up(e, lane);
        unsigned at = seen + inc - e;
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (ordered(element<F32>(v, g * PER + i)) == key && ++at == ties)
            s.cut_id = base + tile_id<F32>(lane, g * PER + i);
        seen += __shfl_sync(0xffffffffu, inc, 31);
      }
    });
  }
  __syncthreads();
  u64 id = tid == 0 && s.cut_id != 0x7fffffff ? (u64)(unsigned)s.cut_id : 0;  // one CTA at most has it
  unsigned any = tid == 0 && s.cut_id != 0x7fffffff;
  r.sum(id, any);
  if (tid == 0) {
    s.cut_key = key;
    s.cut_id = any ? (int)id : 0x7fffffff;
  }
  __syncthreads();
}

template <bool F32, bool VEC, bool SHORT>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(16) unsigned char dyn[];
  Shared& s = *reinterpret_cast<Shared*>(dyn);
  constexpr int WORDS = F32 ? 8 : 4;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = a.nc > 1 ? cluster_ctarank() : 0;
  if (a.nc > 1) cluster_arrive_relaxed();
  const int n = blockIdx.x / a.nc;
  const float T = a.temp ? a.temp[n] : a.temp1, u = a.uniforms[n];
  const float top_p = a.top_p ? a.top_p[n] : a.top_p1, min_p = a.min_p ? a.min_p[n] : a.min_p1;
  const int top_k = a.top_k ? a.top_k[n] : a.top_k1;
  const unsigned K = T == 0.0f ? 1u : top_k > 0 && top_k < a.V ? (unsigned)top_k : 0u;
  const bool by_p = top_p < 1.0f && T > 0.0f, by_m = min_p > 0.0f && T > 0.0f;
  const int begin = min(a.V, (int)rank * a.share), end = min(a.V, begin + a.share);
  const int tiles = (end - begin + kTile - 1) / kTile;
  typedef Entry<SHORT> E;
  typedef typename E::Word Word;
  Row<F32, VEC, SHORT> r{a, s, static_cast<const unsigned char*>(a.logits) + (long long)n * a.stride * (F32 ? 4 : 2),
                  begin, end, tiles, (tiles + kWarps - 1) / kWarps, rank, 0};
  Weigh& w = r.w;

  // Constants of T, in float-floats (fp64 takes longer here than the row).
  float c_hi, c_lo;  // log2(e) / T; c_hi is rounded down and c_lo above 0, so that -inf stays -inf
  const float Tf = T > 0.0f ? T : 1.0f;
  {
    w.unit = __int_as_float(max(254 - (__float_as_int(Tf) >> 23 & 0xff), 1) << 23);
    const float Tu = Tf * w.unit, ih = __fdiv_rn(1.0f, Tu), il = __fmaf_rn(-ih, Tu, 1.0f) * ih;
    w.dc.ih = ih;
    const ff C = ff_mul_f(ff{0x1.62e43p-11f, -0x1.05c61p-39f}, Tu);  // T ln2/1024
    w.dc.ch = C.hi;
    w.dc.cli = C.lo * ih;
    w.dc.inv = __fdiv_rn(1.0f, C.hi);
    w.lmin = -2048.0f * Tu;
    const ff c = ff_mul(ff{0x1.715476p+0f, 0x1.4ae0c0p-26f}, ff{ih, il});
    c_hi = next_down(c.hi);
    c_lo = fmaxf(((c.hi - c_hi) + c.lo) * w.unit, 1e-37f);
    c_hi = fminf(c_hi * w.unit, 0x1p120f);
  }
  if (by_m && warp == kWarps - 1) {  // one warp, since it is fp64
    const double x = (double)(Tf * w.unit) * log((double)min_p);
    if (lane == 0) {
      s.log_hi = (float)x;
      s.log_lo = (float)(x - (double)(float)x);
    }
  }

  // The maximum (NaN if there is one); for top_p alone the sum of all weights, and a sample by value: entries
  // of every step-th tile, or for small k the threads' maxima (where k of them lie, at least k entries do).
  const bool summed = by_p && !K, by_top = K > 1 && K <= 16u * (unsigned)a.nc;
  // Bins of the sample per unit of logit: 16 a power of two of weight, or, where it is the count that matters, 128 for
  // what the row's first 256 entries spread over.
  float unit = 16.0f * c_hi;
  if (K > 1) {
    uint32_t x[WORDS];
    load_tile<F32, VEC>(r.row, 0, a.V, lane, x);
    float top = neg_inf(), low = INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float l = element<F32>(x, e);
      top = fmaxf(top, l);
      if (l > neg_inf()) low = fminf(low, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    // (and so that the bins' edges are floats of their own)
    if (top > low && top - low <= FLT_MAX) unit = fminf(__fdiv_rn(128.0f, top - low), __fdiv_rn(0x1p18f, fmaxf(top, -low)));
  }
  float m = neg_inf();
  // The sum: 2^(n + f - far) for l log2(e)/T = n + f with n whole and |f| <= 1/2, where ex2.approx is off by
  // 1.46e-7 at most (every argument tried), and the roundings of f by 2.1e-8. Eight are added in three steps
  // (2^-24 each) and then in float-floats: the sum is good to 3.5e-7, whatever the entries are (measured: 1.7e-7 at
  // most, 1e-8 for normal logits). far is a thread's maximum so far; entries below lmin count as lmin (2^-101).
  const float reach = -1480.0f * Tf;  // no entry as low as this counts in a row whose sum is used
  float ref = reach, lmin = 1.0475f * reach, far = rintf(reach * c_hi), magic = kRoundMagic - far;
  uint32_t lmin2 = 0;  // the same, two bf16
  if constexpr (!F32) lmin2 = __bfloat16_as_ushort(__float2bfloat16_ru(lmin)) * 0x10001u;
  ff run{0.0f, 0.0f};
  unsigned sampled = 0;
  int to_sample = 1 + warp % a.step;  // tiles of this warp up to the next one that is sampled
  for (int i = tid; i < kValueBins; i += kThreads) s.sample[i] = 0;
  for (int i = tid; i < 1024; i += kThreads) s.tab[i] = kSvExp2Table1024[i];
  for (int i = tid; i < kBins; i += kThreads) s.hlo[i] = s.hhi[i] = s.hcnt[i] = 0;
  if (tid < 2) s.edge[tid] = -1;
  if (tid < 4) s.n_cand[tid] = 0;
  if (tid == 0) {
    s.n_aside = 0;
    s.cut_key = 0;
    s.cut_id = 0x7fffffff;
    s.given = false;
  }
  __syncthreads();
  auto into_sample = [&](float l) {
    // (further than the sample's bins from a maximum so far: far from the row's as well)
    if ((m - l) * unit < (float)kSampleBins) atomicAdd(&s.sample[__float2int_rd(l * unit) & (kValueBins - 1)], 1u);
  };
  if (summed || (K > 1 && !by_top)) {
    r.template all_tiles<F32 ? 2 : 4>([&](int base, const uint32_t (&x)[WORDS]) {
      float top;
      if constexpr (F32) {
        top = __uint_as_float(x[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmax_nan(top, __uint_as_float(x[i]));
      } else {
        const uint32_t t2 = bf16x2_max_nan(bf16x2_max_nan(x[0], x[1]), bf16x2_max_nan(x[2], x[3]));
        top = fmax_nan(bf16_lo(t2), bf16_hi(t2));
      }
      m = fmax_nan(m, top);
      if (summed) {
        if (top > ref) {
          const float to = rintf(top * c_hi), down = __int_as_float(max(127 + __float2int_rn(far - to), 0) << 23);
          run.hi *= down;
          run.lo *= down;
          far = to;
          ref = top;
          magic = kRoundMagic - far;
          lmin = top + 0.0475f * reach;
          if constexpr (!F32) lmin2 = __bfloat16_as_ushort(__float2bfloat16_ru(lmin)) * 0x10001u;
        }
        float2 t2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 l;
          if constexpr (F32) {
            l = make_float2(fmaxf(element<F32>(x, 2 * e), lmin), fmaxf(element<F32>(x, 2 * e + 1), lmin));
          } else {
            const uint32_t l2 = bf16x2_max(x[e], lmin2);
            l = make_float2(bf16_lo(l2), bf16_hi(l2));
          }
          const float2 k = f2_fma(l, f2(c_hi), f2(magic)), n = f2_fma(k, f2(-1.0f), f2(magic));
          const float2 y = f2_fma(l, f2(c_lo), f2_fma(l, f2(c_hi), n));
          t2[e] = make_float2(__uint_as_float(__float_as_uint(ex2_fast(y.x)) + (__float_as_uint(k.x) << 23)),
                              __uint_as_float(__float_as_uint(ex2_fast(y.y)) + (__float_as_uint(k.y) << 23)));
        }
        const float2 t = f2_add(f2_add(t2[0], t2[1]), f2_add(t2[2], t2[3]));
        const ff to = two_sum(run.hi, t.x + t.y);
        run.hi = to.hi;
        run.lo += to.lo;
      }
      if (--to_sample == 0) {
        to_sample = a.step;
        sampled += (unsigned)min(kTile, end - base);
        if (m > neg_inf()) {
#pragma unroll
          for (int e = 0; e < 8; ++e) into_sample(element<F32>(x, e));
        }
      }
    });
  } else {
    uint32_t m2 = 0xff80ff80u;
    r.template all_tiles<F32 ? 4 : 8>([&](int, const uint32_t (&x)[WORDS]) {
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmax_nan(m, __uint_as_float(x[i]));
      } else {
        m2 = bf16x2_max_nan(m2, bf16x2_max_nan(bf16x2_max_nan(x[0], x[1]), bf16x2_max_nan(x[2], x[3])));
      }
    });
    if constexpr (!F32) m = fmax_nan(bf16_lo(m2), bf16_hi(m2));
    if (by_top && m > neg_inf()) into_sample(m);
  }
  // The power of two above the weight of l.
  auto exponent = [&](float l) { return __float2int_rd(fmaxf(fminf(l * w.unit * w.dc.ih * 1.44269504f, 4000.0f), -4000.0f)) + 1; };
  // The CTA's, then the row's; the sum is in whole numbers, as the weights are.
  {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) s.wmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = fmax_nan(m, s.wmax[i]);
    const int e = __float2int_rn(far) - exponent(m) + a.scale_bits;
    u64 sum = summed ? whole(run.hi, e) : 0;
    sum += run.lo < 0.0f ? 0 - whole(-run.lo, e) : whole(run.lo, e);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s.wsum[0][warp] = sum, s.wcnt[0][warp] = sampled;
    __syncthreads();
    if (warp == 0) {
      if (a.nc > 1) cluster_wait();
      sum = 0, sampled = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += s.wsum[0][i], sampled += s.wcnt[0][i];
      if (lane < a.nc) {
        dsmem_st_u32(r.remote(&s.cta_max[rank], lane), __float_as_uint(m));
        dsmem_st_u64(r.remote(&s.cta_sum[rank], lane), sum);
        dsmem_st_u32(r.remote(&s.cta_sampled[rank], lane), sampled);
      }
    } else if (a.nc > 1) {
      cluster_wait();
    }
    r.sync();
    m = s.cta_max[0];
    for (int i = 1; i < a.nc; ++i) m = fmax_nan(m, s.cta_max[i]);
  }

  unsigned fault = 0;
  if (!(m <= FLT_MAX))
    fault = SV_DEV_NONFINITE;
  else if (m == neg_inf())
    fault = SV_DEV_EMPTY_ROW;
  if (!(u >= 0.0f && u <= 1.0f)) fault |= SV_DEV_UNIFORM_RANGE;
  if (!(T >= 0.0f && T <= FLT_MAX) || !(top_p > 0.0f) || !(min_p <= 1.0f)) fault |= SV_DEV_SETTING;
  if (fault) {
    if (rank == 0 && tid == 0) {
      a.out[n] = -1;
      if (a.prob) a.prob[n] = __int_as_float(0x7fc00000);
      if (a.status) atomicOr(a.status, fault);
    }
    return;
  }

  const bool near = fabsf(m * w.unit) < 1386.0f * (Tf * w.unit);
  const bool known = near && T > 1e-30f && T < 1e30f;  // the first pass' sum is good
  // The least logit that min_p keeps: m + T ln(min_p), rounded up; in the weights' unit, since T ln(min_p) may be no fp32
  // number, or a subnormal one.
  float floor_l = -FLT_MAX;
  if (by_m) {
    const float mu = m * w.unit;
    if (fabsf(mu) > 0x1p100f) {
      floor_l = m;  // (every other value is further below than any min_p reaches)
    } else {
      const ff x = two_sum(mu, s.log_hi);
      const ff y = fast_two_sum(x.hi, x.lo + s.log_lo);
      const float least = y.lo > 0.0f ? just_above(y.hi) : y.hi;
      floor_l = __fdiv_rn(least, w.unit);
      if (floor_l * w.unit < least) floor_l = just_above(floor_l);  // (a subnormal that was rounded down)
      floor_l = fmaxf(fminf(floor_l, m), -FLT_MAX);
    }
  }
  {
    w.shift = 44 - a.scale_bits + exponent(near ? m : 0.0f);
    // (so far from m / T that no entry but m counts: a smaller unit does too, and keeps m unit a number)
    if (fabsf(m) * w.unit > 0x1p100f) w.unit = __int_as_float((354 - (__float_as_int(m) >> 23 & 0xff)) << 23);
    w.off = near ? 0.0f : -m * w.unit;
    if (tid == 0) s.w = w;
  }
  const u64 part = by_p ? fraction(top_p) : 0;
  // The least whole mass that is top_p of `total` or more.
  auto part_of = [&](u64 total) { return max(__umul64hi(total, part) + (total * part != 0 ? 1u : 0u), (u64)1); };

  u64 sum = 0;       // a thread's part of the kept mass in the records
  unsigned sure = 0; // entries in them
  bool cut = false;  // s.cut_key and s.cut_id say what is kept of the entries set aside
  float lo = floor_l, hi = just_below(floor_l);

  const bool weigh_all = summed && !known;  // a pass of its own for the mass of all entries
  if ((!K && !by_p) || weigh_all) sum = r.pass(lo, hi, false, weigh_all || !by_m, 0.0f, 0.0f, sure);
  if (K || by_p) {
    bool found = false;
    const u64 w_max = r.weigh(m);
    u64 mass_all = 0;  // of the row
    float mass_f = 0.0f;  // the same, relative to the maximum's
    if (summed) {
      if (weigh_all) {
        unsigned z = 0;
        mass_all = sum;
        r.sum(mass_all, z);
      } else {
        for (int i = 0; i < a.nc; ++i) mass_all += s.cta_sum[i] >> min(exponent(m) - exponent(s.cta_max[i]), 63);
      }
      mass_f = __fdiv_rn(__ull2float_rn(mass_all), __ull2float_rn(w_max));
    }
    const int top_bin = __float2int_rd(m * unit);
    // Edge e of the sample's bins is the value (top_bin - e + 1) / unit, or, where such values are too many for floats
    // (T is small beside m), about the maximum less (e - 1) / unit.
    const bool steep = !(fabsf(m * unit) < 0x1p22f);
    auto edge_at = [&](int e) { return steep ? m - (float)(e - 1) / unit : (float)(top_bin - e + 1) / unit; };
    if (K != 1) {
      unsigned n_sampled = 0;
      for (int i = 0; i < a.nc; ++i) n_sampled += s.cta_sampled[i];
      // Two bins a thread, the deepest first: the sample's mass below, its variance, and the count above.
      const int b = kSampleBins - 2 - 2 * tid, at0 = (int)((unsigned)top_bin - b) & (kValueBins - 1), at1 = (at0 - 1) & (kValueBins - 1);
      unsigned c0 = 0, c1 = 0;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < a.nc) {
          c0 += dsmem_ld_u32(r.remote(&s.sample[at0], i));
          c1 += dsmem_ld_u32(r.remote(&s.sample[at1], i));
        }
      // (a bin's middle is b + part - 1/2 sixteenths below the maximum, part = m unit - top_bin)
      const float mid = (float)b + (steep ? 0.5f : m * unit - (float)top_bin) - 0.5f;
      const float w0 = ex2_fast(-0.0625f * mid), w1 = ex2_fast(-0.0625f * (mid + 1.0f));
      const float m0 = (float)c0 * w0, m1 = (float)c1 * w1, v0 = m0 * w0, v1 = m1 * w1;
      unsigned cc = scan_up(c0 + c1, lane);
      float cm = m0 + m1, cv = v0 + v1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, cm, o), q = __shfl_up_sync(0xffffffffu, cv, o);
        if (lane >= o) cm += y, cv += q;
      }
      if (lane == 31) s.wcnt[1][warp] = cc, s.fmass[warp] = cm, s.fvar[warp] = cv;
      __syncthreads();
      if (a.nc > 1) cluster_arrive_relaxed();  // the other CTAs' samples have been read
      unsigned all_c = 0;
      float below_m = 0.0f, below_v = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) cc += s.wcnt[1][i], below_m += s.fmass[i], below_v += s.fvar[i];
        all_c += s.wcnt[1][i];
      }
      cm += below_m, cv += below_v;
      const float scale = by_top ? 1.0f : (float)a.V / (float)max(n_sampled, 1u);
      const float want_below = K ? 0.0f : (1.0f - top_p) * mass_f / scale;
      int up = -1, down = -1;  // the deepest bin edge that is surely above the cut; that is not surely below it
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int edge = b + j;
        if (K) {
          const float above = (float)(all_c - cc + (j ? c0 : 0u));
          const float dev = by_top ? 0.0f : 3.5f * sqrt_fast(above + 1.0f) + 2.0f;
          if (!by_p && !by_top && (above + dev) * scale <= (float)K) up = edge;
          if ((above - dev) * scale < (float)K) down = edge;
        } else {
          // (An entry that the sample has missed may weigh as much as the edge's: one more in the variance.)
          const float one = j ? w1 : w0, mass = j ? cm - m0 : cm;
          const float dev = 3.5f * sqrt_fast((j ? fmaxf(cv - v0, 0.0f) : cv) + one * one) + 0.03f * mass + 2.0f * one;
          if (mass - dev >= want_below) up = edge;
          if (mass + dev > want_below) down = edge;
        }
      }
      up = __reduce_max_sync(0xffffffffu, up);
      down = __reduce_max_sync(0xffffffffu, down);
      if (lane == 0) {
        atomicMax(&s.edge[0], up);
        atomicMax(&s.edge[1], down);
      }
      if (a.nc > 1) cluster_wait();
      __syncthreads();
    }
    auto next = [&](float from, float to) {
      if (tid == 0) s.given = true, s.next_lo = from, s.next_hi = to;
    };
#pragma unroll 1
    for (int attempt = 0; attempt < 4 && !found; ++attempt) {
      if (attempt > 0) {
        r.sync();  // (what the last attempt left has been read)
        for (int i = tid; i < kBins; i += kThreads) s.hlo[i] = s.hhi[i] = s.hcnt[i] = 0;
        if (tid == 0) s.n_aside = 0;
        if (tid < 4) s.n_cand[tid] = 0;
        __syncthreads();
      }
      if (K == 1) {
        lo = m;
        hi = FLT_MAX;
      } else if (s.given) {
        lo = s.next_lo;
        hi = s.next_hi;
      } else {
        const int wider = 24 * attempt * attempt, up = s.edge[0] - wider, down = s.edge[1] + wider;
        hi = up > 0 ? edge_at(up) : FLT_MAX;
        lo = down + 1 >= kSampleBins ? -FLT_MAX : fmaxf(edge_at(down + 1), -FLT_MAX);
      }
      const bool floored = !(K && by_p) && floor_l >= lo;  // min_p cuts above the window's end
      if (floored) {
        lo = floor_l;
        hi = fmaxf(hi, just_below(floor_l));
      }
      const float top_l = hi == FLT_MAX ? m : hi;
      const float width = s.given ? top_l - lo : fminf(top_l - lo, (float)kSampleBins / unit);
      const float per = width > 0.0f ? (float)kBins / width : 0.0f;
      sum = r.pass(lo, hi, false, false, top_l, per, sure);
      __syncthreads();
      u64 above = sum;
      unsigned above_c = sure, aside = tid == 0 ? s.n_aside : 0u;
      r.sum(above, above_c, aside);
      bool over = false;  // a CTA had no room for all of its window's entries
      for (int i = 0; i < a.nc; ++i) over |= s.inbox_d[~r.turn & 1][i] > r.kAside;
      if (over && (K == 1 || (K && by_p))) break;  // (ties; two cuts, which a narrow window need not both hold)
      const int here = (int)s.n_aside;
      // Masses and counts of the window's bins over all CTAs, two a thread, and what lies above the thread's.
      u64 hm0 = 0, hm1 = 0;
      unsigned hc0 = 0, hc1 = 0;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i)
        if (i < a.nc) {
          const u64 h = dsmem_ld_u64(r.remote(&s.hhi[2 * tid], i)), l = dsmem_ld_u64(r.remote(&s.hlo[2 * tid], i)),
                    c = dsmem_ld_u64(r.remote(&s.hcnt[2 * tid], i));
          hm0 += (h << 32) + (l & 0xffffffffu);
          hm1 += (h >> 32 << 32) + (l >> 32);
          hc0 += (unsigned)c;
          hc1 += (unsigned)(c >> 32);
        }
      u64 im = scan_up(hm0 + hm1, lane), all_m = above;
      unsigned ic = scan_up(hc0 + hc1, lane);
      // (in words of its own, beside the row's sums: those change inboxes, a barrier of all CTAs from one to the next)
      if (lane == 31) s.bins_sum[warp] = im, s.bins_cnt[warp] = ic;
      if (tid == 0) s.bin = -1;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) im += s.bins_sum[i], ic += s.bins_cnt[i];
        all_m += s.bins_sum[i];
      }
      im += above - (hm0 + hm1);
      ic += above_c - (hc0 + hc1);
      const unsigned all_c = above_c + aside;
      int turn = 0;
      bool exact = K || weigh_all;  // the total mass is known exactly
      u64 total = mass_all;
      u64 slack = exact ? 0 : (mass_all >> 22) + (mass_all >> 23) + (unsigned)a.V;  // (a unit a weight, for their rounding)
#pragma unroll 1
      for (int round = K ? 0 : 1; round < 2; ++round) {
        u64 want = K, want_lo = K;
        bool better = false;  // the mass below the window decides, and could be known better
        if (round == 0) {
          if (above_c >= K) {  // the window lies too deep
            if (above_c <= r.kAside) next(hi, FLT_MAX);
            break;
          }
          if (all_c < K) {
            // Fewer than k: all of them are kept, if the window ends where the row or min_p does.
            if (!floored && lo > -FLT_MAX) break;
            total = all_m;
            slack = 0;
            found = !by_p;
            if (found) break;
            continue;
          }
        } else {
          want = part_of(total + slack);
          want_lo = part_of(total - min(slack, total));
          const bool in_sure = above >= want_lo, short_of = all_m < want;
          if (in_sure || short_of) {
            better = !exact && ((in_sure && above < want) || (floored && short_of && all_m >= want_lo));
            if (!better) {
              found = !in_sure && floored;  // min_p cuts first: all entries of the window are kept
              if (in_sure && above_c <= r.kAside) next(hi, FLT_MAX);
              break;
            }
          }
        }
        if (!better) {
          // The bin in which the count or the mass is reached.
          if (turn > 0) {
            if (tid == 0) s.bin = -1;
            r.sync();  // (the last candidates have been read)
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const u64 from = j ? im + hm0 : im, to = from + (j ? hm1 : hm0);
            const unsigned c_from = j ? ic + hc0 : ic, c_to = c_from + (j ? hc1 : hc0);
            if (round == 0 ? c_from < K && c_to >= K : from < want && to >= want) {
              s.bin = 2 * tid + j;
              s.bin_mass = from;
              s.bin_count = c_from;
            }
          }
          __syncthreads();
          const int bin = s.bin;
          if (bin < 0 || turn > 3) break;
          if (over) {  // the bin and its neighbours are the next window
            next(bin < kBins - 1 ? fmaxf(top_l - (float)(bin + 2) / per, lo) : lo,
                 bin > 0 ? top_l - (float)(bin - 1) / per : hi);
            break;
          }
          for (int i = tid; i < here; i += kThreads) {
            const Word e = reinterpret_cast<const Word*>(s.aside)[i];
            const float l = E::value(e);
            if (r.bin_of(l, top_l, per) == bin) {
#pragma unroll 1
              for (int k = 0; k < a.nc; ++k) {
                const unsigned at = dsmem_add_u32(r.remote(&s.n_cand[turn], k), 1u);
                if (at < (unsigned)kCand)
                  dsmem_st_u64(r.remote(&s.cand[at], k), (u64)ordered(l) << 32 | (unsigned)~(begin + E::at(e)));
              }
            }
          }
          r.sync();
          const int n_cand = (int)s.n_cand[turn];
          ++turn;
          if (n_cand > kCand) {
            attempt = 4;  // too many ties
            break;
          }
          order_candidates(s, n_cand, round == 0, want_lo, want);
          __syncthreads();
          const int how = s.cut_found;
          if (how == 0) break;
          better = how == 2 && !exact;
          if (!better) {
            cut = true;
            total = s.cut_mass;
            slack = 0;
            if (round == 1 || !by_p) {
              found = true;
              break;
            }
            continue;
          }
        }
        // The mass below the window, exactly.
        u64 rest = r.below(lo);
        unsigned z = 0;
        r.sum(rest, z);
        total = all_m + rest;
        slack = 0;
        exact = true;
        --round;
      }
      if (found && over) {  // all of the window is kept: the next one is empty, above where it ends
        found = false;
        next(lo, just_below(lo));
      }
    }
    if (found) {
      // What is kept of the entries set aside joins the records.
      const int here = (int)min(s.n_aside, r.kAside);
      const unsigned key = cut ? s.cut_key : 0u;
      const int cut_id = cut ? s.cut_id : 0;
      for (int i = tid; i < here; i += kThreads) {
        const Word e = reinterpret_cast<const Word*>(s.aside)[i];
        const float l = E::value(e);
        const int id = begin + E::at(e);
        const unsigned k = ordered(l);
        if (l >= floor_l && (k > key || (k == key && id <= cut_id))) {
          const u64 x = r.weigh(l);
          const int wp = E::at(e) / kTile / r.seg;
          int j = 0, left = s.recs[wp];  // the first record that ends behind the id
          while (left > 1) {
            const int half = left / 2;
            if (s.rec_end[wp][j + half - 1] <= id)
              j += half, left -= half;
            else
              left = half;
          }
          add64(&s.rec_lo[wp][j], &s.rec_hi[wp][j], x);
          sum += x;
        }
      }
    } else {
      r.sync();
      cut_by_bits(r, K, by_p, part);
      cut = true;
      sum = r.pass(fmaxf(floor_l, unordered(s.cut_key)), FLT_MAX, true, false, 0.0f, 0.0f, sure);
    }
  }

  // The smallest id whose cumulative weight exceeds u times the sum; for u = 1 the last one that is kept.
  const int last_turn = r.turn & 1;
  u64 all = sum;
  unsigned z1 = 0, z2 = 0;
  r.sum(all, z1, z2);
  const u64 goal = u < 1.0f ? __umul64hi(all, fraction(u)) : all - 1;
  u64 before = 0;
#pragma unroll 1
  for (int i = 0; i < (int)rank; ++i) before += s.inbox[last_turn][i];
  if (goal < before || goal >= before + s.inbox[last_turn][rank]) return;
  // Its record, 32 at a time in the order of ids.
  if (warp == 0) {
    int wp = 0;
    u64 start = before;
    int from = begin, to = begin;
    bool there = false;
#pragma unroll 1
    for (int i = 0; i < kWarps * kRecords && !there; i += 32) {
      wp = i / kRecords;
      const int j = i % kRecords + lane, recs = s.recs[wp];
      if (i % kRecords >= recs) continue;
      const u64 x = j < recs ? (u64)s.rec_hi[wp][j] << 32 | s.rec_lo[wp][j] : 0;
      const int e = s.rec_end[wp][min(j, recs - 1)];
      const u64 incl = scan_up(x, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, start + incl > goal);
      if (hit) {
        const int k = __ffs(hit) - 1;
        start += __shfl_sync(0xffffffffu, incl - x, k);
        const int before_e = __shfl_sync(0xffffffffu, e, max(k - 1, 0));
        from = k > 0           ? before_e
               : i % kRecords ? s.rec_end[wp][i % kRecords - 1]
                              : begin + min(tiles, wp * r.seg) * kTile;
        to = __shfl_sync(0xffffffffu, e, k);
        there = true;
      } else {
        start += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (lane == 0) s.hit_from = from, s.hit_to = to, s.hit_start = start;
  }
  __syncthreads();
  // Its tiles, one a warp, until the one that reaches the goal.
  const int from = s.hit_from, to = s.hit_to;
  u64 start = s.hit_start;
  const unsigned key = cut ? s.cut_key : 0u;
  const int cut_id = cut ? s.cut_id : 0;
  float* tile = reinterpret_cast<float*>(s.list[warp]);  // the warp's tile, in the order of ids
  // The kept weight of element 32 i + lane of the tile that begins at `base`.
  auto kept = [&](int i, int base) -> u64 {
    const float l = tile[32 * i + lane];
    const int id = base + 32 * i + lane;
    const unsigned k = ordered(l);
    return l > neg_inf() && l >= floor_l && id >= from && id < to && (k > key || (k == key && id <= cut_id))
               ? r.weigh(l)
               : 0;
  };
  const int t_end = (to - begin + kTile - 1) / kTile;
#pragma unroll 1
  for (int t0 = (from - begin) / kTile; t0 < t_end; t0 += kWarps) {
    const int t = t0 + warp, base = begin + t * kTile;
    uint32_t v[WORDS];
    load_tile<F32, VEC>(r.row, base, t < t_end ? end : 0, lane, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[tile_id<F32>(lane, e)] = element<F32>(v, e);
    __syncwarp();
    u64 x = 0;
    // The first turn sums the warps' tiles; in the second the warp whose tile it is looks for the id.
    u64 run = 0;
    int hit = -1;
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const u64 y = kept(i, base);
        if (turn == 0) {
          x += y;
          continue;
        }
        const u64 incl = scan_up(y, lane);
        const unsigned lanes = __ballot_sync(0xffffffffu, run + incl > goal);
        if (lanes) {
          if (lane == __ffs(lanes) - 1) {
            a.out[n] = base + 32 * i + lane;
            if (a.prob) a.prob[n] = T == 0.0f ? 1.0f : ratio(y, all);
          }
          return;
        }
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
      if (turn == 1) return;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if (lane == 0) s.tile_sum[warp] = x;
      __syncthreads();
      run = start;
#pragma unroll 1
      for (int i = 0; i < kWarps && hit < 0; ++i) {
        if (run + s.tile_sum[i] > goal)
          hit = i;
        else
          run += s.tile_sum[i];
      }
      if (hit != warp) break;
    }
    if (hit >= 0) return;
    start = run;
    __syncthreads();
  }
}

}  // namespace fs
}  // namespace sv

namespace {

template <bool F32, bool VEC, bool SHORT>
int launch(const sv::fs::Args& a, cudaStream_t st) {
  static std::mutex mu;
  static bool set[64] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[device]) {
      if (cudaFuncSetAttribute(sv::fs::sample_kernel<F32, VEC, SHORT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)sizeof(sv::fs::Shared)) != cudaSuccess)
        return SV_ERR_CUDA;
      set[device] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.N * a.nc));
  cfg.blockDim = dim3(sv::fs::kThreads);
  cfg.dynamicSmemBytes = sizeof(sv::fs::Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sv::fs::sample_kernel<F32, VEC, SHORT>, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

using sv::misaligned;

extern "C" int spec_filtered_sample(const void* logits, int64_t row_stride, const float* uniforms, int N, int V,
                                    int dtype, const float* temperatures, float temperature, const int32_t* top_ks,
                                    int top_k, const float* top_ps, float top_p, const float* min_ps, float min_p,
                                    int32_t* out_tokens, float* out_probs, uint32_t* status, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  if (N < 0 || N > (1 << 27) || V < 1 || V > (1 << 30) || (N > 1 && row_stride < V)) return SV_ERR_SHAPE;
  if (!temperatures && !(std::isfinite(temperature) && temperature >= 0.0f)) return SV_ERR_TEMPERATURE;
  if ((!top_ps && !(top_p > 0.0f)) || (!min_ps && !(min_p <= 1.0f))) return SV_ERR_SHAPE;
  if (N == 0) return SV_OK;
  if (!logits || !uniforms || !out_tokens) return SV_ERR_NULL;
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (misaligned(logits, es) || misaligned(uniforms, 4) || misaligned(temperatures, 4) || misaligned(top_ks, 4) ||
      misaligned(top_ps, 4) || misaligned(min_ps, 4) || misaligned(out_tokens, 4) || misaligned(out_probs, 4) ||
      misaligned(status, 4))
    return SV_ERR_ALIGN;
  sv::fs::Args a{};
  a.logits = logits;
  a.stride = row_stride;
  a.uniforms = uniforms;
  a.temp = temperatures;
  a.temp1 = temperature;
  a.top_k = top_ks;
  a.top_k1 = top_k;
  a.top_p = top_ps;
  a.top_p1 = top_p;
  a.min_p = min_ps;
  a.min_p1 = min_p;
  a.N = N;
  a.V = V;
  a.out = out_tokens;
  a.prob = out_probs;
  a.status = status;
  a.nc = 1;
  while (a.nc < sv::fs::kMaxCluster && V >= 8192 * a.nc && ((long long)N * a.nc * 2 <= 608 || V > (dtype == SV_F32 ? 32768 : 65536) * a.nc))
    a.nc *= 2;
  const int tile = sv::fs::kTile;
  a.share = (int)(((long long)V + (long long)tile * a.nc - 1) / ((long long)tile * a.nc) * tile);
  a.step = std::max(1, V / (1 << 14) > 8 ? 8 : V / (1 << 14));
  int lg = 0;
  while ((1ll << lg) < V) ++lg;
  a.scale_bits = std::min(44, 61 - lg);
  const bool vec = !misaligned(logits, 16) && ((size_t)row_stride * es) % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SV_F32) return vec ? launch<true, true, false>(a, st) : launch<true, false, false>(a, st);
  // (more than 524288 ids: long entries, and element loads, since no such vocabulary is common)
  if (a.share > sv::fs::kShortIds) return launch<false, false, false>(a, st);
  return vec ? launch<false, true, true>(a, st) : launch<false, false, true>(a, st);
}
