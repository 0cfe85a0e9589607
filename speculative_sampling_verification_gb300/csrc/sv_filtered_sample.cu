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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 256;       // elements of a warp's step: 8 a lane
constexpr int kChunks = 1024;    // most chunks (of one or more tiles) of a CTA's share
constexpr int kMaxCluster = 8;

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

struct Shared {
  float2 tab1024[1024];
  float2 tab256[256];
  u64 chunk[kChunks];
  unsigned chunk_eq[kChunks];
  u64 wsum[2][kWarps];
  unsigned wcnt[2][kWarps];
  u64 inbox[2][kMaxCluster];
  unsigned inbox_c[2][kMaxCluster];
  float wmax[kWarps];
  unsigned wbad[kWarps];
  int pick;
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

SV_DEVINL unsigned ordered(float f) {
  const unsigned b = __float_as_uint(f + 0.0f);  // -0 is 0
  return b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}

SV_DEVINL u64 weight(float l, const Weigh& w, const Shared& s) {
  ff e;
  if (w.fast) {
    e = exp_draw(fmaxf(l, w.lmin), w.qb, w.dc, s.tab1024);
  } else {
    const ff d = two_sum(l, -w.m);
    if (d.hi == 0.0f) {
      e = {1.0f, 0.0f};
    } else if (!(d.hi > w.low)) {
      e = {0.0f, 0.0f};
    } else {
      const ff p = two_prod(d.hi, w.ih);
      e = exp_ff(p.hi, __fmaf_rn(d.hi, w.il, __fmaf_rn(d.lo, w.ih, p.lo)), s.tab256);
    }
  }
  return (u64)((long long)__float2ll_rn(e.hi * w.scale) + __float2ll_rn(e.lo * w.scale));
}

// Eight elements a lane of the tile at `base` of a row; -inf beyond `end`. Lane and element of an
// id: see tile_id.
template <bool F32, bool VEC>
SV_DEVINL void load_tile(const void* row, int base, int end, int lane, float (&v)[8]) {
  if constexpr (!F32) {
    const int at = base + lane * 8;
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(row) + at;
    if (VEC && at + 8 <= end) {
      const uint4 x = ld_global_nc_v4(p);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = at + i < end ? __bfloat162float(p[i]) : neg_inf();
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int at = base + q * 128 + lane * 4;
      const float* p = static_cast<const float*>(row) + at;
      if (VEC && at + 4 <= end) {
        const uint4 x = ld_global_nc_v4(p);
        v[4 * q] = __uint_as_float(x.x), v[4 * q + 1] = __uint_as_float(x.y);
        v[4 * q + 2] = __uint_as_float(x.z), v[4 * q + 3] = __uint_as_float(x.w);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * q + i] = at + i < end ? p[i] : neg_inf();
      }
    }
  }
}
template <bool F32>
SV_DEVINL int tile_id(int lane, int e) {
  return F32 ? (e >> 2) * 128 + lane * 4 + (e & 3) : lane * 8 + e;
}

// Sums over the row's CTAs, the same in every thread.
struct Joint {
  Shared& s;
  int nc;
  unsigned rank, turn;
  SV_DEVINL void sum(u64& x, unsigned& c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = turn & 1;
    ++turn;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) s.wsum[t][warp] = x, s.wcnt[t][warp] = c;
    __syncthreads();
    x = 0, c = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) x += s.wsum[t][i], c += s.wcnt[t][i];
    if (nc == 1) return;
    if ((int)threadIdx.x < nc) {
      dsmem_st_u64(dsmem_map(smem_u32(&s.inbox[t][rank]), threadIdx.x), x);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                       dsmem_map(smem_u32(&s.inbox_c[t][rank]), threadIdx.x)),
                   "r"(c)
                   : "memory");
    }
    cluster_sync();
    x = 0, c = 0;
    for (int i = 0; i < nc; ++i) x += s.inbox[t][i], c += s.inbox_c[t][i];
  }
};

template <bool F32, bool VEC>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ Args a) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = a.nc > 1 ? cluster_ctarank() : 0;
  if (a.nc > 1) cluster_arrive_relaxed();
  const int n = blockIdx.x / a.nc;
  Joint joint{s, a.nc, rank, 0};
  const float T = a.temp ? a.temp[n] : a.temp1, u = a.uniforms[n];
  const float top_p = a.top_p ? a.top_p[n] : a.top_p1, min_p = a.min_p ? a.min_p[n] : a.min_p1;
  const int top_k = a.top_k ? a.top_k[n] : a.top_k1;
  const void* row = static_cast<const unsigned char*>(a.logits) + (long long)n * a.stride * (F32 ? 4 : 2);
  const int begin = min(a.V, (int)rank * a.share), end = min(a.V, begin + a.share);
  const int tiles = (end - begin + kTile - 1) / kTile, chunks = (tiles + (1 << a.shift) - 1) >> a.shift;
  for (int i = tid; i < 1024; i += kThreads) s.tab1024[i] = kSvExp2Table1024[i];
  if (tid < 256) s.tab256[tid] = kSvExp2Table[tid];

  auto each_tile = [&](auto f) {
    for (int c = warp; c < chunks; c += kWarps)
      for (int t = c << a.shift; t < min(tiles, (c + 1) << a.shift); ++t) {
        float v[8];
        load_tile<F32, VEC>(row, begin + t * kTile, end, lane, v);
        f(c, begin + t * kTile, v);
      }
  };

  // Maximum, NaN and +inf.
  float m = neg_inf();
  bool bad = false;
  each_tile([&](int, int, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m = fmaxf(m, v[i]);
      bad |= !(v[i] <= FLT_MAX);
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s.wmax[warp] = m;
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) m = fmaxf(m, s.wmax[i]);
  if (a.nc > 1) {
    cluster_wait();
    if (tid < a.nc) dsmem_st_u64(dsmem_map(smem_u32(&s.inbox[1][rank]), tid), (u64)ordered(m));
    cluster_sync();
    for (int i = 0; i < a.nc; ++i) {
      const unsigned k = (unsigned)s.inbox[1][i];
      m = fmaxf(m, __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k));
    }
  }
  u64 none = 0;
  unsigned any_bad = bad;
  joint.sum(none, any_bad);

  unsigned fault = 0;
  if (any_bad)
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

  Weigh w;
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
  }
  const unsigned floor_key = ordered(min_p > 0.0f && T > 0.0f
                                         ? fminf(__double2float_ru((double)m + (double)T * log((double)min_p)), m)
                                         : -FLT_MAX);

  // The cut: entries whose key exceeds `cut` are kept, and the first `ties` (by id) of those equal to it.
  unsigned cut = 0, ties = 0xffffffffu;
  const unsigned K = T == 0.0f ? 1u : top_k > 0 && top_k < a.V ? (unsigned)top_k : 0u;
  auto count_mass = [&](unsigned key, bool strict, u64& mass, unsigned& count) {
    u64 x = 0;
    unsigned c = 0;
    each_tile([&](int, int, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const unsigned k = ordered(v[i]);
        if (strict ? k > key : k >= key) {
          ++c;
          x += weight(v[i], w, s);
        }
      }
    });
    joint.sum(x, c);
    mass = x;
    count = c;
  };
  u64 mass;
  unsigned count;
  u64 total = 0;
  if (K) {
    for (int bit = 31; bit >= 0; --bit) {
      count_mass(cut | 1u << bit, false, mass, count);
      if (count >= K) cut |= 1u << bit;
    }
    count_mass(cut, true, mass, count);
    ties = K - count;
    const u64 one = weight(__uint_as_float(cut & 0x80000000u ? cut ^ 0x80000000u : ~cut), w, s);
    total = mass + ties * one;
  }
  if (top_p < 1.0f && T > 0.0f) {
    if (!K) {
      count_mass(0, false, mass, count);
      total = mass;
    }
    const u64 part = (u64)((double)top_p * 18446744073709551616.0);
    const u64 want = max(__umul64hi(total, part) + (total * part != 0 ? 1u : 0u), (u64)1);
    unsigned pcut = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const unsigned tried = pcut | 1u << bit;
      if (tried > cut) {
        count_mass(tried, false, mass, count);
        if (mass >= want) pcut = tried;
      } else {
        pcut = tried;  // the k kept entries reach the whole of the mass
      }
    }
    count_mass(pcut, true, mass, count);
    const u64 one = weight(__uint_as_float(pcut & 0x80000000u ? pcut ^ 0x80000000u : ~pcut), w, s);
    const unsigned need = (unsigned)((want - mass + one - 1) / one);
    ties = pcut > cut ? need : min(ties, need);
    cut = pcut;
  }

  // Entries equal to the cut, by chunk, where not all of them are kept.
  auto kept_of = [&](float l, unsigned& eq_before) -> bool {
    const unsigned k = ordered(l);
    if (k < floor_key || k < cut) return false;
    return k > cut || eq_before < ties;
  };
  for (int i = tid; i < chunks; i += kThreads) s.chunk_eq[i] = 0;
  __syncthreads();
  unsigned eq0 = 0;  // ties in the CTAs before
  if (ties != 0xffffffffu) {
    unsigned mine = 0;
    each_tile([&](int c, int, float (&v)[8]) {
      unsigned e = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) e += ordered(v[i]) == cut;
      e = __reduce_add_sync(0xffffffffu, e);
      if (lane == 0) s.chunk_eq[c] += e;
      mine += lane == 0 ? e : 0;
    });
    const int t = joint.turn & 1;
    u64 z = 0;
    joint.sum(z, mine);
    if (a.nc > 1)
      for (unsigned i = 0; i < rank; ++i) eq0 += s.inbox_c[t][i];
    __syncthreads();
    if (warp == 0) {  // counts before each chunk
      unsigned run = eq0;
      for (int i0 = 0; i0 < chunks; i0 += 32) {
        const unsigned x = i0 + lane < chunks ? s.chunk_eq[i0 + lane] : 0;
        unsigned incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (i0 + lane < chunks) s.chunk_eq[i0 + lane] = run + incl - x;
        run += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
  }
  // Weights of a tile's kept entries, in the order of ids; `eq` counts the ties before it.
  auto kept_weights = [&](float (&v)[8], unsigned& eq, u64 (&x)[8]) {
    constexpr int GROUPS = F32 ? 2 : 1, PER = 8 / GROUPS;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      unsigned mine = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) mine += ordered(v[g * PER + i]) == cut;
      unsigned incl = mine;
      if (ties != 0xffffffffu) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
      }
      unsigned before = eq + incl - mine;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float l = v[g * PER + i];
        x[g * PER + i] = l > neg_inf() && kept_of(l, before) ? weight(l, w, s) : 0;
        before += ordered(l) == cut;
      }
      eq += __shfl_sync(0xffffffffu, incl, 31);
    }
  };

  // Kept weight of every chunk, then the draw.
  u64 mine = 0;
  {
    int last = -1;
    u64 acc = 0;
    unsigned eq = 0;
    each_tile([&](int c, int, float (&v)[8]) {
      if (c != last) {
        acc = 0;
        last = c;
        eq = ties != 0xffffffffu ? s.chunk_eq[c] : 0;
      }
      u64 x[8], sum = 0;
      kept_weights(v, eq, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      acc += sum;
      if (lane == 0) {
        s.chunk[c] = acc;
        mine += sum;
      }
    });
  }
  const int t = joint.turn & 1;
  u64 all = mine;
  unsigned z = 0;
  joint.sum(all, z);
  u64 before = 0;
  u64 here = all;
  if (a.nc > 1) {
    for (unsigned i = 0; i < rank; ++i) before += s.inbox[t][i];
    here = s.inbox[t][rank];
  }
  // The smallest id whose cumulative weight exceeds u times the sum; for u = 1 the last one that is kept.
  const u64 goal = u < 1.0f ? __umul64hi(all, (u64)((double)u * 18446744073709551616.0)) : all - 1;
  if (goal < before || goal >= before + here) return;
  __syncthreads();
  if (warp != 0) return;
  u64 run = before;
  int at = -1;
  for (int i0 = 0; i0 < chunks && at < 0; i0 += 32) {
    const u64 x = i0 + lane < chunks ? s.chunk[i0 + lane] : 0;
    u64 incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal);
    if (hit) {
      const int k = __ffs(hit) - 1;
      at = i0 + k;
      run += __shfl_sync(0xffffffffu, incl - x, k);
    } else {
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  unsigned eq = ties != 0xffffffffu ? s.chunk_eq[at] : 0;
  for (int tl = at << a.shift; tl < min(tiles, (at + 1) << a.shift); ++tl) {
    float v[8];
    load_tile<F32, VEC>(row, begin + tl * kTile, end, lane, v);
    u64 x[8];
    kept_weights(v, eq, x);
    constexpr int GROUPS = F32 ? 2 : 1, PER = 8 / GROUPS;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      u64 sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += x[g * PER + i];
      u64 incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + incl > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          u64 c = run + incl - sum;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (c <= goal && c + x[g * PER + i] > goal) {
              a.out[n] = begin + tl * kTile + tile_id<F32>(lane, g * PER + i);
              if (a.prob) a.prob[n] = T == 0.0f ? 1.0f : (float)((double)x[g * PER + i] / (double)all);
            }
            c += x[g * PER + i];
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

template <bool F32>
int launch(const sv::fs::Args& a, bool vec, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.N * a.nc));
  cfg.blockDim = dim3(sv::fs::kThreads);
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
