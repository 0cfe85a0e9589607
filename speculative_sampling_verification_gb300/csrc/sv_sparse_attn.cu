// Attention over the pages that a cheap score selects for each query
// (sv_sparse_attention), and the bounds of a page's keys that the score is made
// of (sv_page_bounds).
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"
#include "sv_sparse.h"
#include "sv_tree_attn.h"

namespace sv {
namespace sparse {

constexpr float kAmaxMin = 1e-30f;
constexpr float kCodeMax = 127.0f;

// ---------------------------------------------------------------- bounds of a page's keys
//
// For every channel the least and the largest value of a page's keys, as int8 codes
// of one scale for the page and head, rounded outwards: code_min scale <= k_d <=
// code_max scale (to the fp32 rounding of the product that makes the code). A page
// that holds NaN or infinity gets the scale +inf, which selects it before others.
//
// A warp takes a page of a head by itself: its lanes hold a few channels each (8 bytes of a key, 4 or 16
// where those do not fit) and go through the page's keys, several loads under way; no
// barrier, and one exchange at the end. Rows that do not fit (odd or long ones) go channel by channel.

constexpr int kBoundThreads = 128;

struct BoundArgs {
  const void* kc;
  const float* ks;
  long long num_pages;
  int Hkv, D, P, max_pages, B;
  const int32_t *page_table, *ctx_lens, *new_lens;
  int8_t* codes;
  float* scale;
  unsigned* status;
  int chunks;
};

SV_DEVINL float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Of three values in one instruction.
SV_DEVINL float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
SV_DEVINL float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
SV_DEVINL uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

SV_DEVINL signed char bound_code(float x, bool fine) {
  return fine ? (signed char)(int)fminf(fmaxf(x, -kCodeMax), kCodeMax) : (signed char)0;
}

// Four e4m3 codes as floats.
SV_DEVINL void e4m3x4(uint32_t w, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The values in a lane's bytes of a key.
template <bool F8, int BYTES>
struct Piece {
  static constexpr int N = F8 ? BYTES : BYTES / 2;
  uint32_t w[BYTES / 4];
  SV_DEVINL void load(const unsigned char* p) {
    if constexpr (BYTES == 4) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (BYTES == 8) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = v.x, w[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
};

// BYTES a lane (0: any row, channel by channel).
template <bool F8, int BYTES>
__global__ void __launch_bounds__(kBoundThreads) page_bounds_kernel(const __grid_constant__ BoundArgs a) {
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kBoundThreads / 32) + (threadIdx.x >> 5);
  const int hk = (int)(item % a.Hkv), chunk = (int)(item / a.Hkv % a.chunks);
  const long long b = item / a.Hkv / a.chunks;
  if (b >= a.B) return;
  const long long ctx = a.ctx_lens[b], add = a.new_lens[b];
  if (add <= 0) return;
  const long long end = ctx + add;
  if (ctx < 0 || end > (long long)a.max_pages * a.P) {
    if (lane == 0 && a.status) atomicOr(a.status, (unsigned)SV_DEV_PAGE_RANGE);
    return;
  }
  const int p1 = (int)((end + a.P - 1) / a.P);
#pragma unroll 1
  for (int p = (int)(ctx / a.P) + chunk; p < p1; p += a.chunks) {
    const int id = a.page_table[b * a.max_pages + p];
    if (id < 0 || id >= a.num_pages) {
      if (lane == 0 && a.status) atomicOr(a.status, (unsigned)SV_DEV_PAGE_RANGE);
      continue;
    }
    const int count = (int)min((long long)a.P, end - (long long)p * a.P);
    const long long row0 = ((long long)id * a.Hkv + hk) * a.P;
    const long long at = ((long long)id * a.Hkv + hk) * 2 * a.D;
    if constexpr (BYTES > 0) {
      constexpr int N = Piece<F8, BYTES>::N;
      constexpr int U = 64 / BYTES;  // loads under way: 2 KB a warp
      const int row_bytes = F8 ? a.D : 2 * a.D, lanes = row_bytes / BYTES;  // lanes of a key, at most 32
      const int per = 32 / lanes, g = lane / lanes, col = lane - g * lanes;
      const bool on = g < per;
      const unsigned char* base = static_cast<const unsigned char*>(a.kc) + row0 * row_bytes + col * BYTES;
      float lo[N], hi[N];
      uint32_t l2[BYTES / 4], h2[BYTES / 4];
#pragma unroll
      for (int i = 0; i < N; ++i) lo[i] = INFINITY, hi[i] = -INFINITY;
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i) l2[i] = 0x7f807f80u, h2[i] = 0xff80ff80u;
#pragma unroll 1
      for (int r0 = 0; r0 < count; r0 += per * U) {
        Piece<F8, BYTES> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = min(r0 + g + u * per, count - 1);  // (a key twice changes nothing)
          if (on) x[u].load(base + (long long)r * row_bytes);
        }
        // The scales of the turn's keys, a key a lane where 32 lanes have them all.
        const bool spread = per * U <= 32;
        float scale = 0.0f;
        if constexpr (F8) scale = __ldg(a.ks + row0 + min(r0 + lane, count - 1));
        auto scale_of = [&](int u) {
          const int r = g + u * per;
          return spread ? __shfl_sync(0xffffffffu, scale, r & 31) : __ldg(a.ks + row0 + min(r0 + r, count - 1));
        };
#pragma unroll
        for (int u = 0; u < U; u += 2) {
          if constexpr (F8) {
            const float s0 = scale_of(u), s1 = scale_of(u + 1);
#pragma unroll
            for (int q = 0; q < BYTES / 4; ++q) {
              float v[4], z[4];
              e4m3x4(x[u].w[q], v);
              e4m3x4(x[u + 1].w[q], z);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float y = __fmul_rn(v[i], s0), y2 = __fmul_rn(z[i], s1);
                lo[4 * q + i] = min3_nan(lo[4 * q + i], y, y2);
                hi[4 * q + i] = max3_nan(hi[4 * q + i], y, y2);
              }
            }
          } else {
#pragma unroll
            for (int q = 0; q < BYTES / 4; ++q) {
              l2[q] = min2_nan(min2_nan(l2[q], x[u].w[q]), x[u + 1].w[q]);
              h2[q] = bf16x2_max_nan(bf16x2_max_nan(h2[q], x[u].w[q]), x[u + 1].w[q]);
            }
          }
        }
      }
      if constexpr (!F8) {
#pragma unroll
        for (int q = 0; q < BYTES / 4; ++q) {
          lo[2 * q] = bf16_lo(l2[q]), lo[2 * q + 1] = bf16_hi(l2[q]);
          hi[2 * q] = bf16_lo(h2[q]), hi[2 * q + 1] = bf16_hi(h2[q]);
        }
      }
      // The groups of lanes that took different keys of the same channels.
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        for (int k = 1; k < per; ++k) {
          const float y = __shfl_sync(0xffffffffu, lo[i], col + k * lanes), z = __shfl_sync(0xffffffffu, hi[i], col + k * lanes);
          if (g == 0) lo[i] = min_nan(lo[i], y), hi[i] = fmax_nan(hi[i], z);
        }
        if (g == 0) amax = fmax_nan(amax, fmax_nan(fabsf(lo[i]), fabsf(hi[i])));  // |NaN| is NaN
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const bool fine = amax <= FLT_MAX;
      const float top = fmaxf(amax, kAmaxMin), up = __fdiv_rn(kCodeMax, top);
      if (g == 0) {
        signed char c[2][N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          c[0][i] = bound_code(floorf(__fmul_rn(lo[i], up)), fine);
          c[1][i] = bound_code(ceilf(__fmul_rn(hi[i], up)), fine);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          int8_t* to = a.codes + at + (long long)j * a.D + col * N;
#pragma unroll
          for (int i = 0; i < N; i += 2)
            *reinterpret_cast<uint16_t*>(to + i) =
                (uint16_t)((unsigned char)c[j][i] | (unsigned)(unsigned char)c[j][i + 1] << 8);
        }
      }
      if (lane == 0) a.scale[(long long)id * a.Hkv + hk] = fine ? __fdiv_rn(top, kCodeMax) : INFINITY;
    } else {
      // Twice over the channels: the largest magnitude first.
      float amax = 0.0f;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        const bool fine = amax <= FLT_MAX;
        const float top = fmaxf(amax, kAmaxMin), up = __fdiv_rn(kCodeMax, top);
#pragma unroll 1
        for (int d = lane; d < a.D; d += 32) {
          float lo = INFINITY, hi = -INFINITY;
#pragma unroll 4
          for (int r = 0; r < count; ++r) {
            const long long e = (row0 + r) * a.D + d;
            float y;
            if constexpr (F8) {
              const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const unsigned char*>(a.kc)[e], __NV_E4M3);
              y = __fmul_rn(__half2float(*reinterpret_cast<const __half*>(&h)), a.ks[row0 + r]);
            } else {
              y = __bfloat162float(static_cast<const __nv_bfloat16*>(a.kc)[e]);
            }
            lo = min_nan(lo, y);
            hi = fmax_nan(hi, y);
          }
          if (turn == 0) {
            amax = fmax_nan(amax, fmax_nan(fabsf(lo), fabsf(hi)));
          } else {
            a.codes[at + d] = bound_code(floorf(__fmul_rn(lo, up)), fine);
            a.codes[at + a.D + d] = bound_code(ceilf(__fmul_rn(hi, up)), fine);
          }
        }
        if (turn == 0) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        } else if (lane == 0) {
          a.scale[(long long)id * a.Hkv + hk] = fine ? __fdiv_rn(top, kCodeMax) : INFINITY;
        }
      }
    }
  }
}

// ---------------------------------------------------------------- selection
//
// A query row and key/value head are an item, worked on by a cluster of CTAs that
// share its pages. The group's queries become int8 codes (one scale a head), so that
// a page's score is a whole number times two scales: the same whatever the order of
// the sum, and four channels an instruction. sum_d max(q_d min_d, q_d max_d) splits by
// the sign of q: the lanes that hold a page's minima use the negative codes, those that
// hold its maxima the positive ones, and a page is one dot product of 2 D values. The scores go
// as ordered 32-bit keys to the first CTA, which finds the budget-th largest by
// histograms over the keys' range (its least and largest key are known by then), finer until
// the bin's keys are few enough to be ranked one by one, and writes the chosen pages in their order.
// Bound by its chain of steps (table, codes, exchange, histogram, ranks, order), not by its bytes: 24 us alone for 8 heads
// and 8192 pages (17 MB), 21 us for 32 rows and up to 512 pages (22 MB), issue slots 45 % active. With a bisection of the
// keys in place of the histograms the calls took 10 to 16 us longer, and up to 4 us with whole sums in every lane in
// place of sum_lanes.

constexpr int kSelPagesMax = 49152;  // keys of a row in shared memory
constexpr int kSelSmemMax = 212 * 1024;
constexpr unsigned kForced = 0xffffffffu, kInfinite = 0xff800000u;  // keys of forced pages and of +inf
constexpr int kKeyBins = 2048;
constexpr int kSelClusterMax = 16;  // (8 unless the table is too long for it: clusters of 16 do not all fit at once)

struct SelArgs {
  const __nv_bfloat16* q;
  long long q_sn, q_sh;
  const int8_t* codes;
  const float* scale;
  const int32_t *page_table, *positions, *seqs;
  int32_t *selected, *table, *ctx, *parent;
  unsigned *clear, *clear2;  // words that the attention wants at 0
  int clear_words, clear2_words;
  long long num_pages;
  int N, B, Hq, Hkv, D, P, max_pages, budget, sink, recent, nc, ids_cap;
};



SV_DEVINL void dsmem_min_u32(unsigned a, unsigned v) {
  asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
SV_DEVINL void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
SV_DEVINL void cluster_wait_acquire() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

SV_DEVINL void store_key(unsigned keys0, int p, unsigned key, bool cluster) {
  if (cluster)
    dsmem_st_u32(keys0 + p * 4, key);
  else
    asm volatile("st.shared::cta.u32 [%0], %1;" ::"r"(keys0 + p * 4), "r"(key) : "memory");
}

// Sums over the LP lanes of a page of 16 values a lane (16/HC pages of HC heads, in that order): each
// step hands half of the values over to the lane that keeps them, so that a value takes about one exchange. Lane li
// ends up with value li (LP = 16), values 2 li and 2 li + 1 (LP = 8), or value li / 2 (LP = 32).
template <int LP>
SV_DEVINL void sum_lanes(int (&v)[16], int li) {
  int step = LP / 2;
#pragma unroll
  for (int n = 16; n > (LP == 8 ? 2 : 1); n >>= 1, step >>= 1) {
    const bool up = li & step;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const int give = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, step);
    }
  }
  if (LP == 32) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// LP lanes hold the 2 D codes of a page, 16 each (LP = 0: any D, a warp a page); HC heads at a time.
template <int LP, int HC, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : 4) select_kernel(const __grid_constant__ SelArgs a) {
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(16) unsigned char dyn[];
  unsigned* keys = reinterpret_cast<unsigned*>(dyn);               // [max_pages] (first CTA)
  int* ids = reinterpret_cast<int*>(dyn + (size_t)a.max_pages * 4);  // [ids_cap] this CTA's pages
  signed char* qcode = reinterpret_cast<signed char*>(ids + a.ids_cap);  // [HC][Dp]
  __shared__ float qscale[8];
  __shared__ unsigned faults[kSelClusterMax], key_range[2];  // least key, and the largest's complement
  __shared__ int wsum[WARPS], wsum2[WARPS];
  __shared__ __align__(16) unsigned hist[kKeyBins];
  __shared__ unsigned bin_keys[THREADS];
  __shared__ int at_bin[3];  // bin, what is wanted of it, its keys
  __shared__ unsigned n_bin, the_cut;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = a.nc > 1 ? cluster_ctarank() : 0;
  if (tid < 2) key_range[tid] = 0xffffffffu;
  if (tid == 0) n_bin = 0;
  if (a.nc > 1) cluster_arrive();
  const long long item = blockIdx.x / a.nc;
  const int h = (int)(item % a.Hkv);
  const long long n = item / a.Hkv;
  const int G = a.Hq / a.Hkv;
  const int pos = a.positions[n], seq = a.seqs ? a.seqs[n] : (int)n;  // (under way during the codes)
  if (blockIdx.x == 0) {
    for (int i = tid; i < a.clear_words; i += THREADS) a.clear[i] = 0;
    for (int i = tid; i < a.clear2_words; i += THREADS) a.clear2[i] = 0;
  }

  const int Dp = (a.D + 15) & ~15;
  auto codes_of = [&](int h0) {
    // A warp a head: its largest magnitude, then its codes.
    for (int j = warp; j < HC; j += WARPS) {
      float top = 0.0f;
      bool fin = true;
      const __nv_bfloat16* qr = a.q + n * a.q_sn + (long long)(h * G + h0 + j) * a.q_sh;
      const bool on = h0 + j < G;
      for (int d = lane; on && d < a.D; d += 32) {
        const float x = fabsf(__bfloat162float(qr[d]));
        fin = fin && x <= FLT_MAX;
        top = fmaxf(top, x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      fin = __all_sync(0xffffffffu, fin) && on;
      top = fmaxf(top, kAmaxMin);
      const float up = __fdiv_rn(kCodeMax, top);
      for (int d = lane; d < Dp; d += 32) {
        const float x = fin && d < a.D ? rintf(__fmul_rn(__bfloat162float(qr[d]), up)) : 0.0f;
        qcode[j * Dp + d] = (signed char)(int)fminf(fmaxf(x, -kCodeMax), kCodeMax);
      }
      if (lane == 0) qscale[j] = fin ? __fdiv_rn(top, kCodeMax) : 0.0f;
    }
  };
  codes_of(0);  // (nothing else it needs has to be looked up)

  const bool empty = pos == -1 || seq == -1;
  bool fault = !empty && (pos < 0 || (long long)pos >= (long long)a.max_pages * a.P || seq < 0 || seq >= a.B);
  const int np = empty || fault ? 0 : pos / a.P + 1;
  const int K = min(a.budget, np);
  const int32_t* table = a.page_table + (long long)(np ? seq : 0) * a.max_pages;

  // This CTA's pages.
  const int share = (np + a.nc - 1) / a.nc;
  const int first = min(np, (int)rank * share), mine = min(np, first + share) - first;
  bool bad = false;
  for (int i = tid; i < mine; i += THREADS) {
    const int id = table[first + i];
    const bool out = id < 0 || id >= a.num_pages;
    bad |= out;
    ids[i] = out ? 0 : id;
  }
  const bool rank_pages = np > a.budget;  // else all are chosen
  const unsigned keys0 = a.nc > 1 ? dsmem_map(smem_u32(keys), 0) : smem_u32(keys);
  unsigned least = 0xffffffffu, most = 0;  // of this thread's keys, but for the forced pages'

  // The key of page p, this CTA's page i. With more than HC heads the largest so far stays here
  // (rank 0: in its place; there i is p) and goes to the first CTA after the last heads.
  auto put_key = [&](int h0, int i, int p, float best, float ps) {
    const float s = isinf(ps) ? INFINITY : __fmul_rn(best, ps);
    // (NaN, of a scale that was never written, counts as +inf: only forced pages have the key kForced)
    unsigned key = p < a.sink || p >= np - a.recent ? kForced : min(ordered(s), kInfinite);
    if (h0 > 0) key = max(key, keys[i]);
    if (h0 + HC < G) {
      keys[i] = key;
      return;
    }
    store_key(keys0, p, key, a.nc > 1);
    if (key != kForced) {
      least = min(least, key);
      most = max(most, key);
    }
  };
  auto joined = [&] {  // this CTA's pages are known, and the first CTA is there
    bad = __syncthreads_or(bad);
    if (a.nc > 1) cluster_wait_acquire();
  };

  if (rank_pages) {
#pragma unroll 1
    for (int h0 = 0; h0 < G; h0 += HC) {
      if (h0) __syncthreads();
      if (h0 > 0) codes_of(h0);
      if (h0 == 0)
        joined();
      else
        __syncthreads();
      if constexpr (LP > 0) {
        constexpr int PPW = 32 / LP, U = 16 / HC;  // pages of a load; loads of a turn
        const int li = lane % LP, sub = lane / LP, half = a.D / 16;
        const bool used = li < 2 * half, upper = li >= half;
        const int off = (upper ? li - half : li) * 16;
        int qv[HC][4];
#pragma unroll
        for (int j = 0; j < HC; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const unsigned w = used ? *reinterpret_cast<const unsigned*>(qcode + j * Dp + off + 4 * k) : 0u;
            const unsigned neg = __vcmpgtu4(w & 0x80808080u, 0u);  // bytes below zero
            qv[j][k] = (int)(upper ? w & ~neg : w & neg);
          }
        // The value that sum_lanes leaves in this lane: page my_u of the turn, head my_j (LP = 8: and the next).
        const int value = LP == 8 ? 2 * li : LP == 16 ? li : li / 2, my_u = value / HC, my_j = value % HC;
        const bool there = h0 + my_j < G, there1 = h0 + my_j + 1 < G;
        const float qs0 = qscale[my_j], qs1 = LP == 8 ? qscale[my_j + 1] : 0.0f;
        const int stride = a.Hkv * 2 * a.D;
        const int8_t* base = a.codes + (long long)h * 2 * a.D + li * 16;
        auto fetch = [&](int i0, uint4 (&c)[U], float& ps) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int id = ids[min(i0 + u * PPW + sub, mine - 1)];
            c[u] = used ? __ldg(reinterpret_cast<const uint4*>(base + (long long)id * stride)) : make_uint4(0, 0, 0, 0);
          }
          ps = __ldg(a.scale + (long long)ids[min(i0 + my_u * PPW + sub, mine - 1)] * a.Hkv + h);
        };
        uint4 c[U], ahead[U];  // the next turn's pages are under way while one is worked on
        float ps, ps_ahead = 0.0f;
        int i0 = warp * PPW * U;
        if (i0 < mine) fetch(i0, ahead, ps_ahead);
#pragma unroll 1
        for (; i0 < mine; i0 += WARPS * PPW * U) {
#pragma unroll
          for (int u = 0; u < U; ++u) c[u] = ahead[u];
          ps = ps_ahead;
          if (i0 + WARPS * PPW * U < mine) fetch(i0 + WARPS * PPW * U, ahead, ps_ahead);
          const int i = i0 + my_u * PPW + sub;
          int v[16];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < HC; ++j) {
              int s = __dp4a((int)c[u].x, qv[j][0], 0);
              s = __dp4a((int)c[u].y, qv[j][1], s);
              s = __dp4a((int)c[u].z, qv[j][2], s);
              v[u * HC + j] = __dp4a((int)c[u].w, qv[j][3], s);
            }
          sum_lanes<LP>(v, li);
          float best = there ? __fmul_rn((float)v[0], qs0) : -INFINITY;
          if (LP == 8) best = fmaxf(best, there1 ? __fmul_rn((float)v[1], qs1) : -INFINITY);
          // The other heads' lanes.
#pragma unroll
          for (int o = LP == 32 ? 2 : 1; o < (LP == 8 ? HC / 2 : LP == 16 ? HC : 2 * HC); o <<= 1)
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
          if (my_j == 0 && (LP != 32 || !(li & 1)) && i < mine) put_key(h0, i, first + i, best, ps);
        }
      } else {
        for (int i = warp; i < mine; i += WARPS) {
          const int p = first + i;
          const long long at = (long long)ids[i] * a.Hkv + h;
          float best = -INFINITY;
          for (int j = 0; j < HC && h0 + j < G; ++j) {
            int s = 0;
            for (int d = lane; d < a.D; d += 32) {
              const int x = qcode[j * Dp + d];
              s += x * (int)a.codes[at * 2 * a.D + (x > 0 ? a.D : 0) + d];
            }
            s = __reduce_add_sync(0xffffffffu, s);
            best = fmaxf(best, __fmul_rn((float)s, qscale[j]));
          }
          if (lane == 0) {
            put_key(h0, i, p, best, a.scale[at]);
          }
        }
      }
    }
  }
  if (rank_pages) {
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      dsmem_min_u32(a.nc > 1 ? dsmem_map(smem_u32(&key_range[0]), 0) : smem_u32(&key_range[0]), least);
      dsmem_min_u32(a.nc > 1 ? dsmem_map(smem_u32(&key_range[1]), 0) : smem_u32(&key_range[1]), ~most);
    }
  } else {
    joined();
  }
  if (tid == 0) {
    if (a.nc > 1)
      dsmem_st_u32(dsmem_map(smem_u32(&faults[rank]), 0), bad);
    else
      faults[0] = bad;
  }
  if (a.nc > 1) cluster_sync();
  if (rank != 0) return;
  __syncthreads();
  for (int i = 0; i < a.nc; ++i) fault = fault || faults[i] != 0;

  int32_t* sel = a.selected ? a.selected + item * a.budget : nullptr;
  int32_t* out = a.table + item * a.budget;
  const int take = fault ? 0 : K;
  if (h == 0 && tid == 0) {
    // The chosen pages' keys as a context of their own: the last page is always
    // chosen and ends with the query's own key.
    a.ctx[n] = fault ? -1 : empty ? 0 : (K - 1) * a.P + pos % a.P;
    a.parent[n] = empty ? -2 : -1;
  }
  for (int i = take + tid; i < a.budget; i += THREADS) {
    if (sel) sel[i] = -1;
    out[i] = -1;
  }
  if (take == 0) return;
  if (!rank_pages) {
    for (int i = tid; i < take; i += THREADS) {
      if (sel) sel[i] = i;
      out[i] = table[i];
    }
    return;
  }
  // The K-th largest key.
  unsigned cut = kForced, from = key_range[0], range = ~key_range[1] - from;
  int need = K - a.sink - a.recent;  // of the keys from `from` to from + range; the forced ones are above
#pragma unroll 1
  while (need > 0) {
    const int shift = max(0, 21 - __clz(range));  // fewer than 2048 bins
    for (int i = tid; i < kKeyBins; i += THREADS) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < np; i += THREADS) {
      const unsigned k = keys[i];
      if (k != kForced && k - from <= range) atomicAdd(&hist[(k - from) >> shift], 1u);
    }
    __syncthreads();
    // A few bins a thread, the largest keys first.
    constexpr int BINS = kKeyBins / THREADS;
    const int b0 = kKeyBins - BINS - BINS * tid;
    unsigned c[BINS];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < BINS; ++i) {
      c[i] = hist[b0 + BINS - 1 - i];
      sum += (int)c[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += z;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    for (int i = 0; i < warp; ++i) incl += wsum[i];
    int above = incl - sum;
    if (above < need && incl >= need) {
#pragma unroll
      for (int i = 0; i < BINS; ++i) {
        if (above < need && above + (int)c[i] >= need) {
          at_bin[0] = b0 + BINS - 1 - i;
          at_bin[1] = need - above;
          at_bin[2] = (int)c[i];
        }
        above += (int)c[i];
      }
    }
    __syncthreads();
    const unsigned bin = (unsigned)at_bin[0];
    need = at_bin[1];
    const int few = at_bin[2];
    if (shift == 0) {
      cut = from + bin;
      break;
    }
    from += bin << shift;
    range = (1u << shift) - 1u;
    if (few <= THREADS) {
      for (int i = tid; i < np; i += THREADS) {
        const unsigned k = keys[i];
        if (k != kForced && k - from <= range) bin_keys[atomicAdd(&n_bin, 1u)] = k;
      }
      __syncthreads();
      if (tid < few) {
        const unsigned k = bin_keys[tid];
        int gt = 0, ge = 0;
        for (int i = 0; i < few; ++i) {
          gt += bin_keys[i] > k;
          ge += bin_keys[i] >= k;
        }
        if (gt < need && ge >= need) the_cut = k;
      }
      __syncthreads();
      cut = the_cut;
      break;
    }
  }
  // Keys above the cut, and the first of those equal to it. A warp takes a run of pages.
  const int run = (np + WARPS - 1) / WARPS;
  const int r0 = min(np, warp * run), r1 = min(np, r0 + run);
  int above = 0, equal = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    above += keys[i] > cut;
    equal += keys[i] == cut;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  __syncthreads();
  if (lane == 0) {
    wsum[warp] = above;
    wsum2[warp] = equal;
  }
  __syncthreads();
  int all_above = 0, above0 = 0, equal0 = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    if (i < warp) {
      above0 += wsum[i];
      equal0 += wsum2[i];
    }
    all_above += wsum[i];
  }
  const int ties = K - all_above;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const unsigned key = i < r1 ? keys[i] : 0u;
    const bool gt = i < r1 && key > cut, eq = i < r1 && key == cut;
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    const unsigned below = (1u << lane) - 1;
    const int ng = above0 + __popc(bg & below), ne = equal0 + __popc(be & below);
    if (gt || (eq && ne < ties)) {
      const int to = ng + min(ne, ties);
      if (sel) sel[to] = i;
      out[to] = table[i];
    }
    above0 += __popc(bg);
    equal0 += __popc(be);
  }
}

// ---------------------------------------------------------------- host side

struct Layout {
  size_t off_table, off_ctx, off_parent, off_counters, off_ml, off_o, total;
  int splits;
};

bool sizes_ok(int N, int Hq, int Hkv, int D, int max_pages, int page_size, int budget) {
  // The chosen pages are a page table of `budget` entries a head to the attention.
  return tat::sizes_ok(N, 1, Hq, Hkv, D, max_pages, page_size) && max_pages <= kSelPagesMax && budget >= 1 &&
         tat::sizes_ok(N, 1, Hq, Hkv, D, budget, page_size) && (long long)N * Hkv < (1ll << 27);
}

Layout make_layout(int N, int Hq, int Hkv, int D, int page_size, int budget) {
  Layout L{};
  size_t off = align_up(sv_tree_attention_workspace_size(N, 1, Hq, Hkv, D, budget, page_size), 256);
  L.off_table = off;
  off = align_up(off + (size_t)N * Hkv * budget * 4, 256);
  L.off_ctx = off;
  off = align_up(off + (size_t)N * 4, 256);
  L.off_parent = off;
  off = align_up(off + (size_t)N * 4, 256);
  // For the few-rows kernel: parts of an item that have arrived, and their results.
  if (dec::takes(Hq / Hkv, D, page_size)) {
    L.splits = dec::splits_of((long long)N * Hkv, budget, page_size);
    const size_t parts = (size_t)dec::most_parts((long long)N * Hkv, budget, page_size) * (Hq / Hkv);
    L.off_counters = off;
    off = align_up(off + (size_t)N * Hkv * 4, 256);
    L.off_ml = off;
    off = align_up(off + parts * 8, 256);
    L.off_o = off;
    off = align_up(off + parts * D * 4, 256);
  }
  L.total = off;
  return L;
}

template <int LP, int HC, int THREADS>
int launch_select_of(const SelArgs& a, size_t smem, cudaStream_t st) {
  static std::mutex mu;
  static bool set[64] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[device]) {
      if (cudaFuncSetAttribute(select_kernel<LP, HC, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelSmemMax) !=
              cudaSuccess ||
          cudaFuncSetAttribute(select_kernel<LP, HC, THREADS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return SV_ERR_CUDA;
      set[device] = true;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.N * a.Hkv * a.nc));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.nc;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel<LP, HC, THREADS>, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

// Large CTAs where there are too few to fill the SMs with small ones.
template <int LP, int HC>
int launch_select(const SelArgs& a, size_t smem, cudaStream_t st) {
  constexpr int kLarge = HC == 4 ? 1024 : 512;
  if ((long long)a.N * a.Hkv * a.nc <= 152 && a.max_pages >= 256 * a.nc) return launch_select_of<LP, HC, kLarge>(a, smem, st);
  return launch_select_of<LP, HC, 256>(a, smem, st);
}

int launch_select_any(SelArgs& a, cudaStream_t st) {
  // CTAs of an item: as many as one wave holds with few items, and no fewer than 64 pages each.
  const long long items = (long long)a.N * a.Hkv;
  a.nc = 1;
  while (a.nc < 8 && items * a.nc * 2 <= 608 && a.max_pages >= 128 * a.nc) a.nc *= 2;
  const int G = a.Hq / a.Hkv, hc = G <= 4 ? 4 : 8;
  size_t smem;
  for (;; a.nc *= 2) {  // (tables so long that a CTA cannot hold an item's keys and pages are shared in any case)
    a.ids_cap = ((a.max_pages + a.nc - 1) / a.nc + 3) & ~3;
    smem = (size_t)((a.max_pages + 3) & ~3) * 4 + (size_t)a.ids_cap * 4 + (size_t)hc * ((a.D + 15) & ~15);
    if (smem <= kSelSmemMax) break;
    if (a.nc == kSelClusterMax) return SV_ERR_SHAPE;
  }
  const int lp = a.D % 16 || a.D > 256 || misaligned(a.codes, 16) ? 0 : a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  if (hc == 4) {
    switch (lp) {
      case 8: return launch_select<8, 4>(a, smem, st);
      case 16: return launch_select<16, 4>(a, smem, st);
      case 32: return launch_select<32, 4>(a, smem, st);
      default: return launch_select<0, 4>(a, smem, st);
    }
  }
  switch (lp) {
    case 8: return launch_select<8, 8>(a, smem, st);
    case 16: return launch_select<16, 8>(a, smem, st);
    case 32: return launch_select<32, 8>(a, smem, st);
    default: return launch_select<0, 8>(a, smem, st);
  }
}

}  // namespace sparse
}  // namespace sv

using namespace sv::sparse;
using sv::misaligned;

extern "C" {

int sv_page_bounds(const void* k_cache, const float* k_scale, int64_t num_pages, int page_size, int cache_dtype,
                   const int32_t* page_table, const int32_t* ctx_lens, const int32_t* new_lens, int B, int Hkv,
                   int D, int max_pages, int8_t* codes, float* scale, uint32_t* status, void* stream) {
  if (cache_dtype != SV_BF16 && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (B < 0 || Hkv < 1 || D < 1 || D > sv::kHeadDimMax || max_pages < 1 || page_size < 1 || num_pages < 1 ||
      num_pages > (1ll << 31) || (long long)max_pages * page_size >= (1ll << 31) || (long long)B * Hkv >= (1ll << 27))
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!k_cache || !page_table || !ctx_lens || !new_lens || !codes || !scale) return SV_ERR_NULL;
  if (cache_dtype == SV_E4M3 && !k_scale) return SV_ERR_NULL;
  if (misaligned(k_cache, cache_dtype == SV_BF16 ? 2 : 1) || misaligned(page_table, 4) || misaligned(ctx_lens, 4) ||
      misaligned(new_lens, 4) || misaligned(scale, 4) || misaligned(status, 4) ||
      (cache_dtype == SV_E4M3 && misaligned(k_scale, 4)))
    return SV_ERR_ALIGN;
  BoundArgs a{};
  a.kc = k_cache;
  a.ks = k_scale;
  a.num_pages = num_pages;
  a.Hkv = Hkv;
  a.D = D;
  a.P = page_size;
  a.max_pages = max_pages;
  a.B = B;
  a.page_table = page_table;
  a.ctx_lens = ctx_lens;
  a.new_lens = new_lens;
  a.codes = codes;
  a.scale = scale;
  a.status = status;
  // Warps for 48 a SM: the pages of a (sequence, head) are shared among them. With few items, whose new
  // tokens may be a long prompt's, a warp for each of up to 1024 pages, so that the warps' loads even out.
  const long long items = (long long)B * Hkv;
  a.chunks = (int)std::max(1ll, std::min((long long)max_pages, std::max(7296 / items, items <= 64 ? 1024ll : 1ll)));
  const bool f8 = cache_dtype == SV_E4M3;
  // The bytes of a lane: 32 lanes hold a row, whose pieces are aligned and even in number of codes.
  const int row = f8 ? D : 2 * D;
  // 8 bytes rather than 4 where both would do (a prompt of 128 thousand e4m3 tokens, 8 heads of 128: 38 us against 44).
  int bytes = 0;
  for (int w : {16, 4, 8})
    if (row % w == 0 && row / w <= 32 && !misaligned(k_cache, w) && !misaligned(codes, 2) && D % 2 == 0) bytes = w;
  const unsigned grid = (unsigned)((items * a.chunks + kBoundThreads / 32 - 1) / (kBoundThreads / 32));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (f8) {
    if (bytes == 4) page_bounds_kernel<true, 4><<<grid, kBoundThreads, 0, st>>>(a);
    else if (bytes == 8) page_bounds_kernel<true, 8><<<grid, kBoundThreads, 0, st>>>(a);
    else if (bytes == 16) page_bounds_kernel<true, 16><<<grid, kBoundThreads, 0, st>>>(a);
    else page_bounds_kernel<true, 0><<<grid, kBoundThreads, 0, st>>>(a);
  } else {
    if (bytes == 4) page_bounds_kernel<false, 4><<<grid, kBoundThreads, 0, st>>>(a);
    else if (bytes == 8) page_bounds_kernel<false, 8><<<grid, kBoundThreads, 0, st>>>(a);
    else if (bytes == 16) page_bounds_kernel<false, 16><<<grid, kBoundThreads, 0, st>>>(a);
    else page_bounds_kernel<false, 0><<<grid, kBoundThreads, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

size_t sv_sparse_attention_workspace_size(int N, int Hq, int Hkv, int D, int max_pages, int page_size, int budget) {
  if (!sizes_ok(N, Hq, Hkv, D, max_pages, page_size, budget)) return 0;
  return make_layout(N, Hq, Hkv, D, page_size, budget).total;
}

int sv_sparse_attention(const void* q, int64_t q_stride_n, int64_t q_stride_h, const void* k_cache,
                        const void* v_cache, const float* k_scale, const float* v_scale, int64_t num_pages,
                        int page_size, int cache_dtype, const int8_t* codes, const float* bound_scale,
                        const int32_t* page_table, const int32_t* positions, const int32_t* seqs, int N, int B,
                        int Hq, int Hkv, int D, int max_pages, int budget, int sink, int recent, float scale,
                        void* out, int32_t* selected, void* workspace, size_t workspace_bytes, void* stream) {
  if (cache_dtype != SV_BF16 && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (!sizes_ok(N, Hq, Hkv, D, max_pages, page_size, budget) || B < 0 || num_pages < 1 || num_pages > (1ll << 31) ||
      sink < 0 || recent < 1 || (long long)sink + recent > budget || !std::isfinite(scale) || !(scale > 0.0f))
    return SV_ERR_SHAPE;
  if (N == 0) return SV_OK;
  if (!seqs && N > B) return SV_ERR_SHAPE;
  if (!q || !k_cache || !v_cache || !codes || !bound_scale || !page_table || !positions || !out || !workspace)
    return SV_ERR_NULL;
  if (cache_dtype == SV_E4M3 && (!k_scale || !v_scale)) return SV_ERR_NULL;
  const size_t ces = cache_dtype == SV_BF16 ? 2 : 1;
  if (misaligned(q, 2) || misaligned(out, 2) || misaligned(k_cache, ces) || misaligned(v_cache, ces) ||
      misaligned(bound_scale, 4) || misaligned(page_table, 4) || misaligned(positions, 4) || misaligned(seqs, 4) ||
      misaligned(selected, 4) || misaligned(workspace, 256) ||
      (cache_dtype == SV_E4M3 && (misaligned(k_scale, 4) || misaligned(v_scale, 4))))
    return SV_ERR_ALIGN;
  const Layout L = make_layout(N, Hq, Hkv, D, page_size, budget);
  if (workspace_bytes < L.total) return SV_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SelArgs s{};
  s.q = static_cast<const __nv_bfloat16*>(q);
  s.q_sn = q_stride_n;
  s.q_sh = q_stride_h;
  s.codes = codes;
  s.scale = bound_scale;
  s.page_table = page_table;
  s.positions = positions;
  s.seqs = seqs;
  s.selected = selected;
  s.table = reinterpret_cast<int32_t*>(ws + L.off_table);
  s.ctx = reinterpret_cast<int32_t*>(ws + L.off_ctx);
  s.parent = reinterpret_cast<int32_t*>(ws + L.off_parent);
  s.clear = reinterpret_cast<unsigned*>(ws);
  const bool few = L.splits > 0 && !misaligned(q, 16) && !misaligned(k_cache, 16) && !misaligned(v_cache, 16) &&
                   q_stride_n % 8 == 0 && q_stride_h % 8 == 0;
  s.clear_words = few ? 1 : (int)sv::tat::cleared_words(1, Hq, Hkv, D, page_size);
  s.clear2 = reinterpret_cast<unsigned*>(ws + L.off_counters);
  s.clear2_words = few ? N * Hkv : 0;
  s.num_pages = num_pages;
  s.N = N;
  s.B = B;
  s.Hq = Hq;
  s.Hkv = Hkv;
  s.D = D;
  s.P = page_size;
  s.max_pages = max_pages;
  s.budget = budget;
  s.sink = sink;
  s.recent = recent;
  const int rc = launch_select_any(s, st);
  if (rc != SV_OK) return rc;
  if (few) {
    sv::sparse::dec::Args d{};
    d.q = s.q;
    d.q_sn = q_stride_n;
    d.q_sh = q_stride_h;
    d.kc = k_cache;
    d.vc = v_cache;
    d.ks = k_scale;
    d.vs = v_scale;
    d.table = s.table;
    d.ctx = s.ctx;
    d.parent = s.parent;
    d.out = static_cast<__nv_bfloat16*>(out);
    d.status = static_cast<unsigned*>(workspace);
    d.counters = s.clear2;
    d.part_ml = reinterpret_cast<float2*>(ws + L.off_ml);
    d.part_o = reinterpret_cast<float*>(ws + L.off_o);
    d.N = N;
    d.Hq = Hq;
    d.Hkv = Hkv;
    d.D = D;
    d.P = page_size;
    d.budget = budget;
    d.splits = L.splits;
    d.scale = scale;
    return sv::sparse::dec::launch(d, cache_dtype, st);
  }
  sv::tat::Args a{};
  a.q = s.q;
  a.q_sb = q_stride_n;
  a.q_st = 0;
  a.q_sh = q_stride_h;
  a.kc = k_cache;
  a.vc = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.page_table = s.table;
  a.ctx_lens = s.ctx;
  a.parents = s.parent;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<unsigned*>(workspace);
  a.num_pages = num_pages;
  a.B = N;
  a.T = 1;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.P = page_size;
  a.max_pages = budget;
  a.table_heads = Hkv;
  a.chained = 1;
  a.scale = scale;
  return sv::tat::launch_attention(a, cache_dtype, workspace, st);
}

}  // extern "C"
