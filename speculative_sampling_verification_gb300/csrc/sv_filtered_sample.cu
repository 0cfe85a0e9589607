// Sampling with temperature, top-k, top-p and min-p from given uniforms
// (spec_filtered_sample): one token a row, from the softmax of the entries that a row's
// own settings keep.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace fs {

typedef unsigned long long u64;

// The kept entries are a prefix of the row in the order of logits, so that a row needs its
// cut: the last entry that is kept. A cluster of CTAs shares a row and passes over it, the first time
// from memory and then from L2:
//   1. the maximum;
//   2. a sample of the tiles, as counts by distance from the maximum, which gives a value that the
//      cut is expected to lie above (a window), with room to spare;
//   3. the entries of the window go to lists in shared memory, 32 at a time to be weighed by full
//      warps; the weights below it, wanted for the mass that top_p is a part of, are summed in
//      fp32. A histogram of the listed entries (counts and masses) gives the cut's bin, the first CTA
//      orders that bin's entries and finds the cut among them;
//   4. the kept entries' masses by chunk of ids, the chunk that the uniform falls in, and its token.
// All decisions are made on whole-number masses (2^-44 of the largest weight). Where the fp32 sum below
// the window could change the cut, that sum is made again with the exact weights; where
// the window turns out too small, it is widened; a row that still has no cut, or too many entries
// in the cut's bin (ties), is halved bit by bit over the keys, with a pass for every bit.

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 256;       // elements of a warp's step: 8 a lane
constexpr int kChunks = 1024;    // most chunks (of one or more tiles) of a CTA's share
constexpr int kMaxCluster = 8;
constexpr int kBins = 512;       // bins of the window
constexpr int kSampleBins = 256; // bins of the sample, 1/8 of a power of two each
constexpr int kList = 256;       // listed entries of a warp
constexpr int kCand = 1024;      // entries of the cut's bin
constexpr int kSampled = 16384;  // elements of a row's sample

struct Args {
  const void* logits;
  long long stride;
  const float* uniforms;
  const float *temp, *top_p, *min_p;
  const int32_t* top_k;
  float temp1, top_p1, min_p1;
  int top_k1;
  int N, V, nc, share, shift, scale_bits;
  int32_t* out;
  float* prob;
  unsigned* status;
};

struct Cut {
  unsigned key;  // entries of a larger key are kept, and those of this key up to `id`
  int id;
  u64 mass;      // of the kept entries
  int found;
};

// What a row's weights are made of: w(l) = exp((l - m)/T) times a power of two, as a whole
// number of 2^-scale_bits (so that sums do not depend on their order).
struct Weigh {
  bool fast;
  int qb;
  DrawConst dc;
  float ih, il, m, lmin, low;
  float scale;
};

struct Shared {
  float2 tab[1024];
  float lv[kWarps][kList];
  int li[kWarps][kList];
  union {
    u64 cand[kCand];                                  // key, then ~id: entries of the cut's bin
    struct { unsigned lo[kChunks], hi[kChunks]; } ch; // kept mass by chunk
    unsigned eq[kChunks];                             // ties by chunk
  };
  unsigned hlo[kBins], hhi[kBins], hcnt[kBins];
  unsigned sample[kSampleBins];
  u64 wsum[2][kWarps];
  unsigned wcnt[2][kWarps];
  u64 inbox[2][kMaxCluster];
  unsigned inbox_c[2][kMaxCluster];
  float wmax[kWarps];
  unsigned ncand[2];
  unsigned listed[kWarps];
  int over, bin;
  u64 bin_mass;
  unsigned bin_count;
  Cut cut;
  Weigh w;
};

SV_DEVINL unsigned ordered(float f) {
  const unsigned b = __float_as_uint(f + 0.0f);  // -0 is 0
  return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}
SV_DEVINL float unordered(unsigned k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The weight for rows whose maximum is too far from 0 for the short exponential.
__device__ __noinline__ u64 weight_far(float l, float m, float ih, float il, float low, float scale) {
  const ff d = two_sum(l, -m);
  ff e{1.0f, 0.0f};
  if (d.hi != 0.0f) {
    if (!(d.hi > low)) return 0;
    const ff p = two_prod(d.hi, ih);
    e = exp_ff(p.hi, __fmaf_rn(d.hi, il, __fmaf_rn(d.lo, ih, p.lo)), kSvExp2Table);
  }
  return (u64)((long long)__float2ll_rn(e.hi * scale) + __float2ll_rn(e.lo * scale));
}

SV_DEVINL u64 weight(float l, const Weigh& w, const Shared& s) {
  if (!w.fast) return weight_far(l, w.m, w.ih, w.il, w.low, w.scale);
  const ff e = exp_draw(fmaxf(l, w.lmin), w.qb, w.dc, s.tab);
  return (u64)((long long)__float2ll_rn(e.hi * w.scale) + __float2ll_rn(e.lo * w.scale));
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

SV_DEVINL uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
SV_DEVINL float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
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
SV_DEVINL void dsmem_st_u32(unsigned a, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
SV_DEVINL unsigned dsmem_add_u32(unsigned a, unsigned v) {
  unsigned r;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(r) : "r"(a), "r"(v) : "memory");
  return r;
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

template <bool F32, bool VEC>
struct Row {
  const Args& a;
  Shared& s;
  const void* row;
  int begin, end, tiles, chunks;
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

  // Sums over the row's CTAs, the same in every thread; `before`: over the CTAs of lower rank, `mine`: this one's.
  SV_DEVINL void sum(u64& x, unsigned& c, u64* before = nullptr, u64* mine = nullptr, unsigned* c_before = nullptr) {
    const int t = turn & 1;
    ++turn;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane() == 0) s.wsum[t][threadIdx.x >> 5] = x, s.wcnt[t][threadIdx.x >> 5] = c;
    __syncthreads();
    x = 0, c = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) x += s.wsum[t][i], c += s.wcnt[t][i];
    if (before) *before = 0, *mine = x;
    if (c_before) *c_before = 0;
    if (a.nc == 1) return;
    if ((int)threadIdx.x < a.nc) {
      dsmem_st_u64(remote(&s.inbox[t][rank], threadIdx.x), x);
      dsmem_st_u32(remote(&s.inbox_c[t][rank], threadIdx.x), c);
    }
    cluster_sync();
    x = 0, c = 0;
    for (int i = 0; i < a.nc; ++i) {
      if (i == (int)rank) {
        if (before) *before = x;
        if (c_before) *c_before = c;
      }
      x += s.inbox[t][i], c += s.inbox_c[t][i];
    }
  }

  // f(chunk, first id, words) for the tiles of this CTA's share, U at a time loaded ahead; a warp takes whole chunks.
  template <int U, typename F>
  SV_DEVINL void tiles_by_chunk(F f) {
    const int per = 1 << a.shift, wp = warp();
    // The warp's tiles as one sequence: i -> chunk wp + (i / per) * kWarps.
    const int n_chunks = chunks > wp ? (chunks - wp + kWarps - 1) / kWarps : 0, n = n_chunks << a.shift;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += U) {
      uint32_t x[U][F32 ? 8 : 4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u, t = ((wp + (i >> a.shift) * kWarps) << a.shift) + (i & (per - 1));
        load_tile<F32, VEC>(row, begin + t * kTile, i < n && t < tiles ? end : 0, lane(), x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u, c = wp + (i >> a.shift) * kWarps, t = (c << a.shift) + (i & (per - 1));
        if (i < n && t < tiles) f(c, begin + t * kTile, x[u]);
      }
    }
  }
  // The same in any order of tiles.
  template <int U, typename F>
  SV_DEVINL void any_tiles(F f, int first = 0, int step = 1) {
    const int stride = kWarps * step;
#pragma unroll 1
    for (int t0 = first + warp() * step; t0 < tiles; t0 += stride * U) {
      uint32_t x[U][F32 ? 8 : 4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = t0 + u * stride;
        load_tile<F32, VEC>(row, begin + t * kTile, t < tiles ? end : 0, lane(), x[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + u * stride < tiles) f(begin + (t0 + u * stride) * kTile, x[u]);
    }
  }

  // Largest element of a lane's eight (no NaN among them).
  SV_DEVINL float top_of(const uint32_t (&x)[F32 ? 8 : 4]) {
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

  // The entries l >= lo of this CTA's share, each once, to f(l, id), by full warps; the lists
  // keep them all unless s.over is set. `tile(words)` sees every tile first.
  template <typename G, typename F>
  SV_DEVINL void scan_above(float lo, G tile, F f) {
    const int ln = lane(), wp = warp();
    float* lv = s.lv[wp];
    int* li = s.li[wp];
    int n = 0;
    bool full = false;
    any_tiles<F32 ? 2 : 4>([&](int base, const uint32_t (&x)[F32 ? 8 : 4]) {
      tile(x);
      if (!__any_sync(0xffffffffu, top_of(x) >= lo)) return;
      unsigned mask = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) mask |= element<F32>(x, e) >= lo ? 1u << e : 0u;
      const unsigned c = __popc(mask), incl = scan_up(c, ln), all = __shfl_sync(0xffffffffu, incl, 31);
      if (n + (int)all > kList) {
        full = true;
        __syncwarp();
        for (int i = ln; i < n; i += 32) f(lv[i], li[i]);
        n = 0;
        __syncwarp();
      }
      int at = n + (int)(incl - c);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (mask >> e & 1u) {
          lv[at] = element<F32>(x, e);
          li[at] = base + tile_id<F32>(ln, e);
          ++at;
        }
      n += (int)all;
    });
    __syncwarp();
    for (int i = ln; i < n; i += 32) f(lv[i], li[i]);
    if (ln == 0) {
      s.listed[wp] = n;
      if (full) s.over = 1;
    }
  }
  // The listed entries again, or those l >= lo by another pass.
  template <typename F>
  SV_DEVINL void again(float lo, F f) {
    if (s.over) {
      scan_above(lo, [](const uint32_t (&)[F32 ? 8 : 4]) {}, f);
    } else {
      const int wp = warp();
      for (int i = lane(); i < (int)s.listed[wp]; i += 32) f(s.lv[wp][i], s.li[wp][i]);
    }
  }
};

// Among the n candidates of the cut's bin (first CTA), the one at which the running count reaches
// `want_count`, or the running mass `want` (and does so for every mass from want_lo to want).
// s.bin_mass and s.bin_count are what lies above the bin.
__device__ __noinline__ void order_candidates(Shared& s, int n, bool by_count, u64 want_lo, u64 want) {
  const int tid = threadIdx.x;
  if (tid == 0) s.cut.found = 0;
  int size = 32;
  while (size < n) size <<= 1;
  for (int i = n + tid; i < size; i += kThreads) s.cand[i] = 0;
  __syncthreads();
  // Largest first (bitonic).
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = tid; i < size / 2; i += kThreads) {
        const int p = (i / j) * 2 * j + i % j, q = p + j;
        const u64 x = s.cand[p], y = s.cand[q];
        const bool down = (p & k) == 0;
        if (down ? x < y : x > y) s.cand[p] = y, s.cand[q] = x;
      }
      __syncthreads();
    }
  // One warp adds the weights up, 32 at a time.
  if (tid >= 32) return;
  u64 mass = s.bin_mass;
  const unsigned above_count = s.bin_count;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const u64 c = i0 + tid < n ? s.cand[i0 + tid] : 0;
    const u64 x = i0 + tid < n ? weight(unordered((unsigned)(c >> 32)), s.w, s) : 0;
    const u64 incl = scan_up(x, tid);
    const bool hit = i0 + tid < n &&
                     (by_count ? above_count + i0 + tid + 1 == want : mass + incl >= want && mass + incl - x < want);
    if (hit) {
      s.cut.key = (unsigned)(c >> 32);
      s.cut.id = (int)~(unsigned)c;
      s.cut.mass = mass + incl;
      s.cut.found = by_count || mass + incl - x < want_lo ? 1 : 2;
    }
    mass += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <bool F32, bool VEC>
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
  const int begin = min(a.V, (int)rank * a.share), end = min(a.V, begin + a.share);
  const int tiles = (end - begin + kTile - 1) / kTile;
  Row<F32, VEC> r{a, s, static_cast<const unsigned char*>(a.logits) + (long long)n * a.stride * (F32 ? 4 : 2),
                  begin, end, tiles, (tiles + (1 << a.shift) - 1) >> a.shift, rank, 0};
  Weigh& w = r.w;

  // Maximum (NaN if there is one).
  float m = neg_inf();
  {
    uint32_t m2 = 0xff80ff80u;
    r.template any_tiles<F32 ? 4 : 8>([&](int, const uint32_t (&x)[WORDS]) {
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max_nan(m, __uint_as_float(x[i]));
      } else {
        m2 = max2_nan(m2, max2_nan(max2_nan(x[0], x[1]), max2_nan(x[2], x[3])));
      }
    });
    if constexpr (!F32) m = max_nan(bf16_lo(m2), bf16_hi(m2));
  }
  for (int i = tid; i < 1024; i += kThreads) s.tab[i] = kSvExp2Table1024[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s.wmax[warp] = m;
  for (int i = tid; i < kSampleBins; i += kThreads) s.sample[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) m = max_nan(m, s.wmax[i]);
  if (a.nc > 1) {
    cluster_wait();
    if (tid < a.nc) dsmem_st_u32(r.remote(&s.inbox_c[1][rank], tid), __float_as_uint(m));
    cluster_sync();
    for (int i = 0; i < a.nc; ++i) m = max_nan(m, __uint_as_float(s.inbox_c[1][i]));
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

  float c_hi, c_lo, far, tail_unit;  // a weight is about tail_unit 2^(l (c_hi + c_lo) - far)
  {
    const double Td = T > 0.0f ? (double)T : 1.0, inv = 1.0 / Td, C = Td * 0.69314718055994530942 / 1024.0;
    w.ih = (float)inv;
    w.il = (float)(inv - (double)w.ih);
    w.dc.ch = (float)C;
    w.dc.cli = (float)((C - (double)w.dc.ch) * inv);
    w.dc.inv = (float)(1.0 / C);
    w.dc.ih = w.ih;
    w.m = m;
    const double top = (double)m * inv;
    w.fast = fabs(top) < 1386.0;
    w.qb = 127 - ((int)floor((w.fast ? top : 0.0) * 1.4426950408889634074) + 1);
    w.lmin = (float)(-2048.0 * Td);
    w.low = (float)(-88.0 * Td);
    w.scale = __int_as_float((127 + a.scale_bits) << 23);
    // c_hi is c rounded down and c_lo above 0, so that -inf stays -inf.
    const double c = 1.4426950408889634074 * inv;
    c_hi = __double2float_rd(c);
    c_lo = fmaxf((float)(c - (double)c_hi), 1e-37f);
    far = (float)((double)m * c);
    if (tid == 0) s.w = w;
    tail_unit = (float)((double)weight(m, w, s) * exp2((double)far - (double)m * c));
  }
  const float floor_l = min_p > 0.0f && T > 0.0f
                            ? fminf(__double2float_ru((double)m + (double)T * log((double)min_p)), m)
                            : -FLT_MAX;
  const unsigned K = T == 0.0f ? 1u : top_k > 0 && top_k < a.V ? (unsigned)top_k : 0u;
  const bool by_p = top_p < 1.0f && T > 0.0f;
  const u64 part = (u64)((double)(by_p ? top_p : 0.0f) * 18446744073709551616.0);
  // The least whole mass that is top_p of `total` or more.
  auto part_of = [&](u64 total) { return max(__umul64hi(total, part) + (total * part != 0 ? 1u : 0u), (u64)1); };

  Cut cut{0, 0x7fffffff, 0, 1};  // everything
  float lo = floor_l;            // the lists hold the entries l >= lo
  bool lists = false;

  if (K || by_p) {
    bool found = false;
    const float unit = 8.0f * c_hi;  // sample bins per unit of logit
    if (K != 1 && w.fast) {
      const int step = max(1, a.V / kSampled);
      r.template any_tiles<2>(
          [&](int, const uint32_t (&x)[WORDS]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float d = (m - element<F32>(x, e)) * unit;
              if (d < (float)kSampleBins) atomicAdd(&s.sample[(int)d], 1u);
            }
          },
          0, step);
      r.sync();
      unsigned c = 0;
      for (int i = 0; i < a.nc; ++i) c += dsmem_ld_u32(r.remote(&s.sample[tid], i));
      // Running count and mass from the top, a bin a thread.
      const float mass1 = (float)c * ex2_fast(-0.125f * ((float)tid + 0.5f));
      unsigned cc = scan_up(c, lane);
      float cm = mass1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, cm, o);
        if (lane >= o) cm += y;
      }
      if (lane == 31) s.wcnt[0][warp] = cc, s.wmax[warp] = cm;
      __syncthreads();
      float all = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) cc += s.wcnt[0][i], cm += s.wmax[i];
        all += s.wmax[i];
      }
      // Kept for the attempts below: counts as they are, masses as parts of the sample's.
      s.hcnt[tid] = cc;
      s.hlo[tid] = __float_as_uint(all - cm + 1e-6f * all);  // mass below the bin
      s.hhi[tid] = __float_as_uint(all);
      r.sync();
    }
    int edge_k = 0, edge_p = 0;
    // The window's lower end, from the sample; -FLT_MAX where it does not reach far enough.
    if (K == 1) {
      lo = m;
    } else if (!w.fast) {
      lo = -FLT_MAX;
    }
#pragma unroll 1
    for (int attempt = 0; attempt < 3 && !found; ++attempt) {
      if (K != 1 && w.fast) {
        if (attempt == 0) {
          // Bins that hold enough of the sample: searched by all threads at once.
          const int step = max(1, a.V / kSampled);
          const float need = K ? (1.25f * (float)K + 12.0f * sqrtf((float)K) + 40.0f) / (float)step : 0.0f;
          const float all = __uint_as_float(s.hhi[tid]);
          const float spare = 0.5f * (1.0f - top_p) * all;
          const bool short_k = K && (float)s.hcnt[tid] < need;
          const bool short_p = !K && by_p && __uint_as_float(s.hlo[tid]) > spare;
          edge_k = __syncthreads_count(short_k);
          edge_p = __syncthreads_count(short_p);
        } else {
          edge_k += 16 * attempt * attempt;
          edge_p += 12 * attempt * attempt;
        }
        const int edge = max(edge_k, edge_p) + 1;
        lo = edge >= kSampleBins ? -FLT_MAX : fmaxf(m - (float)edge / unit, -FLT_MAX);
      }
      const bool floored = !(K && by_p) && floor_l >= lo;  // min_p cuts above the window's end
      if (floored) lo = floor_l;
      if (attempt > 0)
        r.sync();  // the last attempt's bins have been read
      else
        __syncthreads();
      for (int i = tid; i < kBins; i += kThreads) s.hlo[i] = s.hhi[i] = s.hcnt[i] = 0;
      if (tid < 2) s.ncand[tid] = 0;
      if (tid == 0) s.over = 0;
      __syncthreads();
      const float width = fminf(m - lo, 256.0f / unit);  // (32 powers of two; further down is the last bin's)
      const float per = width > 0.0f ? (float)kBins / width : 0.0f;
      auto bin_of = [&](float l) { return min(kBins - 1, (int)fminf((m - l) * per, (float)kBins)); };
      // Masses below the window: fp32, eight at a time, then lane by lane as whole numbers.
      const bool tail = by_p && !K;
      u64 tail_mass = 0;
      auto into_bins = [&](float l, int) {
        const int b = bin_of(l);
        add64(&s.hlo[b], &s.hhi[b], weight(l, w, s));
        atomicAdd(&s.hcnt[b], 1u);
      };
      if (tail) {
        float run = 0.0f;
        r.scan_above(
            lo,
            [&](const uint32_t (&x)[WORDS]) {
              float t8 = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 l = make_float2(element<F32>(x, e), element<F32>(x, e + 1));
                const float2 y = f2_fma(l, f2(c_lo), f2_fma(l, f2(c_hi), f2(-far)));
                const float p = l.x >= lo ? 0.0f : ex2_fast(y.x), q = l.y >= lo ? 0.0f : ex2_fast(y.y);
                t8 += p + q;
              }
              run += t8;
            },
            into_bins);
        tail_mass = (u64)((double)run * (double)tail_unit);
      } else {
        r.scan_above(lo, [](const uint32_t (&)[WORDS]) {}, into_bins);
      }
      lists = true;
      unsigned z = 0;
      r.sum(tail_mass, z);  // (its barrier completes the bins)
      __syncthreads();
      // All CTAs' bins, two a thread, and what lies above each.
      u64 hm[2] = {0, 0};
      unsigned hc[2] = {0, 0};
      for (int i = 0; i < a.nc; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int b = 2 * tid + j;
          hm[j] += (u64)dsmem_ld_u32(r.remote(&s.hhi[b], i)) << 32 | 0;
          hm[j] += dsmem_ld_u32(r.remote(&s.hlo[b], i));
          hc[j] += dsmem_ld_u32(r.remote(&s.hcnt[b], i));
        }
      u64 im = scan_up(hm[0] + hm[1], lane);
      unsigned ic = scan_up(hc[0] + hc[1], lane);
      const int t = r.turn & 1;
      ++r.turn;
      if (lane == 31) s.wsum[t][warp] = im, s.wcnt[t][warp] = ic;
      __syncthreads();
      u64 all_m = 0;
      unsigned all_c = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) im += s.wsum[t][i], ic += s.wcnt[t][i];
        all_m += s.wsum[t][i], all_c += s.wcnt[t][i];
      }
      im -= hm[0] + hm[1];  // above this thread's two bins
      ic -= hc[0] + hc[1];
      u64 total = all_m + tail_mass;
      u64 slack = tail_mass >> 20;  // what the fp32 sum may be off by
      bool again_exact = false;
#pragma unroll 1
      for (int round = K ? 0 : 1; round < (by_p ? 2 : 1); ++round) {
        const bool count = round == 0;
        if (count && all_c < K) {
          // Fewer entries than k: with the floor inside the window it cuts; else the window is too small.
          if (floored || lo == -FLT_MAX) found = true;
          break;
        }
        if (!count && K) total = cut.mass, slack = 0;
        const u64 want = count ? (u64)K : part_of(total + slack);
        const u64 want_lo = count ? (u64)K : part_of(total - slack);
        if (!count && all_m < want) {
          if (floored && all_m < want_lo) {
            found = true;  // the floor cuts first
            cut = Cut{0, 0x7fffffff, 0, 1};
            break;
          }
          if (!floored && lo > -FLT_MAX && !K) break;  // the window is too small
        }
        // The bin in which the count or the mass is reached.
        if (tid == 0) s.bin = -1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const u64 m0 = im + (j ? hm[0] : 0), m1 = m0 + hm[j];
          const unsigned c0 = ic + (j ? hc[0] : 0), c1 = c0 + hc[j];
          if (count ? c0 < K && c1 >= K : m0 < want && m1 >= want) {
            s.bin = 2 * tid + j;
            s.bin_mass = m0;
            s.bin_count = c0;
          }
        }
        __syncthreads();
        const int bin = s.bin;
        if (bin < 0) break;
        r.again(lo, [&](float l, int id) {
          if (bin_of(l) == bin) {
            const unsigned at = dsmem_add_u32(r.remote(&s.ncand[round], 0), 1u);
            if (at < (unsigned)kCand)
              dsmem_st_u64(r.remote(&s.cand[at], 0), (u64)ordered(l) << 32 | (unsigned)~id);
          }
        });
        r.sync();
        if (rank == 0) {
          __syncthreads();
          const int nc = (int)s.ncand[round];
          if (nc <= kCand)
            order_candidates(s, nc, count, want_lo, want);
          else if (tid == 0)
            s.cut.found = 0;
          __syncthreads();
        }
        r.sync();
        cut.found = (int)dsmem_ld_u32(r.remote(&s.cut.found, 0));
        cut.key = dsmem_ld_u32(r.remote(&s.cut.key, 0));
        cut.id = (int)dsmem_ld_u32(r.remote(&s.cut.id, 0));
        cut.mass = dsmem_ld_u64(r.remote(&s.cut.mass, 0));
        if (cut.found == 2 && !again_exact) {
          // The fp32 sum decides nothing here: the mass below the window once more, exactly.
          u64 rest = 0;
          r.template any_tiles<1>([&](int, const uint32_t (&x)[WORDS]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float l = element<F32>(x, e);
              if (l < lo && l > neg_inf()) rest += weight(l, w, s);
            }
          });
          r.sum(rest, z);
          total = all_m + rest;
          slack = 0;
          again_exact = true;
          if (tid == 0) s.ncand[round] = 0;
          r.sync();
          --round;
          continue;
        }
        if (cut.found != 1) {
          attempt = 3;  // ties: bit by bit
          break;
        }
        if (round == (by_p ? 1 : 0)) found = true;
      }
    }
    if (!found) {
      // Bit by bit over the keys: the largest key that the wanted count or mass reaches, then the last of its
      // ties that is kept.
      auto reach = [&](unsigned key, u64& mass, unsigned& count) {  // entries of this key or more
        u64 x = 0;
        unsigned c = 0;
        r.template any_tiles<2>([&](int, const uint32_t (&v)[WORDS]) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float l = element<F32>(v, e);
            if (l > neg_inf() && ordered(l) >= key) {
              ++c;
              x += weight(l, w, s);
            }
          }
        });
        r.sum(x, c);
        mass = x;
        count = c;
      };
      u64 mass = 0, total = 0;
      unsigned count = 0, ties = 0xffffffffu, key = 0;
      if (K) {
        for (int bit = 31; bit >= 0; --bit) {
          reach(key | 1u << bit, mass, count);
          if (count >= K) key |= 1u << bit;
        }
        reach(key + 1, mass, count);
        ties = K - count;
        total = key ? mass + ties * weight(unordered(key), w, s) : mass;
      }
      if (by_p) {
        if (!K) {
          reach(0, mass, count);
          total = mass;
        }
        const u64 want = part_of(total);
        unsigned pkey = 0;
        for (int bit = 31; bit >= 0; --bit) {
          const unsigned tried = pkey | 1u << bit;
          if (tried <= key) {
            pkey = tried;  // the k kept entries reach all of their mass
          } else {
            reach(tried, mass, count);
            if (mass >= want) pkey = tried;
          }
        }
        reach(pkey + 1, mass, count);
        const u64 one = weight(unordered(pkey), w, s);
        const u64 need = one ? (want - mass + one - 1) / one : 1;
        ties = pkey > key ? (unsigned)need : (unsigned)min((u64)ties, need);
        key = pkey;
      }
      // The id of the last tie that is kept: ties by chunk, then within the chunk.
      __syncthreads();
      for (int i = tid; i < kChunks; i += kThreads) s.eq[i] = 0;
      __syncthreads();
      unsigned mine = 0, ties_before = 0;
      r.template tiles_by_chunk<1>([&](int c, int, const uint32_t (&v)[WORDS]) {
        unsigned e = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) e += ordered(element<F32>(v, i)) == key;
        e = __reduce_add_sync(0xffffffffu, e);
        if (lane == 0) {
          s.eq[c] += e;
          mine += e;
        }
      });
      u64 z = 0;
      unsigned all_eq = mine;
      r.sum(z, all_eq, nullptr, nullptr, &ties_before);
      __syncthreads();
      cut = Cut{key, 0x7fffffff, 0, 1};
      if (tid == 0) s.cut.id = 0x7fffffff;
      __syncthreads();
      if (all_eq > ties && warp == 0) {
        // Does the tie number `ties` lie here?
        unsigned run = ties_before;
        for (int i0 = 0; i0 < r.chunks; i0 += 32) {
          const unsigned x = i0 + lane < r.chunks ? s.eq[i0 + lane] : 0, incl = scan_up(x, lane);
          const unsigned hit = __ballot_sync(0xffffffffu, run + incl >= ties && run + incl - x < ties);
          if (hit) {
            const int k = __ffs(hit) - 1, c = i0 + k;
            unsigned seen = run + __shfl_sync(0xffffffffu, incl - x, k);
            for (int tl = c << a.shift; tl < min(tiles, (c + 1) << a.shift); ++tl) {
              uint32_t v[WORDS];
              load_tile<F32, VEC>(r.row, begin + tl * kTile, end, lane, v);
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
                    s.cut.id = begin + tl * kTile + tile_id<F32>(lane, g * PER + i);
                seen += __shfl_sync(0xffffffffu, inc, 31);
              }
            }
            break;
          }
          run += __shfl_sync(0xffffffffu, incl, 31);
        }
      }
      __syncthreads();
      u64 id = (u64)(unsigned)(s.cut.id == 0x7fffffff ? 0 : s.cut.id + 1);  // one CTA at most has it
      if (tid != 0) id = 0;
      unsigned any = tid == 0 && s.cut.id != 0x7fffffff;
      r.sum(id, any);
      if (any) cut.id = (int)id - 1;
      lo = fmaxf(floor_l, fmaxf(unordered(key), -FLT_MAX));
      lists = false;
    }
  }

  // Masses of the kept entries by chunk.
  const bool all_kept = cut.key == 0 && floor_l == -FLT_MAX;
  auto kept = [&](float l, int id) {
    const unsigned k = ordered(l);
    return l >= floor_l && (k > cut.key || (k == cut.key && id <= cut.id));
  };
  __syncthreads();
  for (int i = tid; i < kChunks; i += kThreads) s.ch.lo[i] = s.ch.hi[i] = 0;
  if (!lists && tid == 0) s.over = 1;
  __syncthreads();
  u64 sum = 0;
  if (all_kept) {
    r.template tiles_by_chunk<1>([&](int c, int, const uint32_t (&x)[WORDS]) {
      u64 t8 = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float l = element<F32>(x, e);
        t8 += l > neg_inf() ? weight(l, w, s) : 0;
      }
      sum += t8;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t8 += __shfl_xor_sync(0xffffffffu, t8, o);
      if (lane == 0) add64(&s.ch.lo[c], &s.ch.hi[c], t8);
    });
  } else {
    const float from = cut.key ? fmaxf(lo, fmaxf(floor_l, unordered(cut.key))) : fmaxf(lo, floor_l);
    r.again(from, [&](float l, int id) {
      if (kept(l, id)) {
        const u64 x = weight(l, w, s);
        const int c = (id - begin) / kTile >> a.shift;
        add64(&s.ch.lo[c], &s.ch.hi[c], x);
        sum += x;
      }
    });
  }
  u64 all = sum, before = 0, here = 0;
  unsigned z = 0;
  r.sum(all, z, &before, &here);
  // The smallest id whose cumulative weight exceeds u times the sum; for u = 1 the last one that is kept.
  const u64 goal = u < 1.0f ? __umul64hi(all, (u64)((double)u * 18446744073709551616.0)) : all - 1;
  if (goal < before || goal >= before + here) return;
  __syncthreads();
  if (warp != 0) return;
  u64 run = before;
  int at = -1;
  for (int i0 = 0; i0 < r.chunks && at < 0; i0 += 32) {
    const u64 x = i0 + lane < r.chunks ? (u64)s.ch.hi[i0 + lane] << 32 | s.ch.lo[i0 + lane] : 0;
    const u64 incl = scan_up(x, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal);
    if (hit) {
      const int k = __ffs(hit) - 1;
      at = i0 + k;
      run += __shfl_sync(0xffffffffu, incl - x, k);
    } else {
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (at < 0) return;
  for (int tl = at << a.shift; tl < min(tiles, (at + 1) << a.shift); ++tl) {
    uint32_t v[WORDS];
    load_tile<F32, VEC>(r.row, begin + tl * kTile, end, lane, v);
#pragma unroll
    for (int g = 0; g < (F32 ? 2 : 1); ++g) {
      constexpr int PER = F32 ? 4 : 8;
      u64 x[PER], part8 = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float l = element<F32>(v, g * PER + i);
        x[i] = l > neg_inf() && kept(l, begin + tl * kTile + tile_id<F32>(lane, g * PER + i)) ? weight(l, w, s) : 0;
        part8 += x[i];
      }
      const u64 incl = scan_up(part8, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          u64 c = run + incl - part8;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (c <= goal && c + x[i] > goal) {
              a.out[n] = begin + tl * kTile + tile_id<F32>(lane, g * PER + i);
              if (a.prob) a.prob[n] = T == 0.0f ? 1.0f : (float)((double)x[i] / (double)all);
            }
            c += x[i];
          }
        }
        return;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

}  // namespace fs
}  // namespace sv

namespace {

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

static_assert(sizeof(sv::fs::Shared) <= 48 * 1024, "shared memory");

template <bool F32>
int launch(const sv::fs::Args& a, bool vec, cudaStream_t st) {
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
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, sv::fs::sample_kernel<F32, true>, a)
                            : cudaLaunchKernelEx(&cfg, sv::fs::sample_kernel<F32, false>, a);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

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
  while (a.nc < sv::fs::kMaxCluster && (long long)N * a.nc * 2 <= 608 && V >= 8192 * a.nc) a.nc *= 2;
  const int tile = sv::fs::kTile;
  a.share = (int)(((long long)V + (long long)tile * a.nc - 1) / ((long long)tile * a.nc) * tile);
  while ((long long)tile << a.shift < ((long long)a.share + sv::fs::kChunks - 1) / sv::fs::kChunks) ++a.shift;
  int lg = 0;
  while ((1ll << lg) < V) ++lg;
  a.scale_bits = std::min(44, 61 - lg);
  const bool vec = !misaligned(logits, 16) && ((size_t)row_stride * es) % 16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SV_F32 ? launch<true>(a, vec, st) : launch<false>(a, vec, st);
}
