// The two memory-bound steps before a tree's attention: queries and keys
// normalised per head and rotated by their positions in one pass
// (sv_qk_norm_rope), and the paged key/value cache, quantised as it is written
// and read back (sv_cache_write, sv_cache_read).
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace tio {

constexpr int kThreads = 128;
constexpr int kSms = 152;

// ---------------------------------------------------------------- element access

// VEC consecutive elements of a row as fp32 (bf16: VEC = 8, fp32: VEC = 4, one
// 16-byte load; VEC = 1: one element).
template <int DT, int VEC>
SV_DEVINL void load_vec(const void* base, long long at, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = DT == SV_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at])
                         : static_cast<const float*>(base)[at];
  } else if constexpr (DT == SV_BF16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(x[i]);
      v[2 * i + 1] = bf16_hi(x[i]);
    }
  } else {
    const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    v[0] = w.x;
    v[1] = w.y;
    v[2] = w.z;
    v[3] = w.w;
  }
}

SV_DEVINL uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The one rounding to the output's type, to nearest even.
template <int DT, int VEC>
SV_DEVINL void store_vec(void* base, long long at, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if (DT == SV_BF16)
      static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v[0]);
    else
      static_cast<float*>(base)[at] = v[0];
  } else if constexpr (DT == SV_BF16) {
    uint4 w;
    w.x = pack_bf16(v[0], v[1]);
    w.y = pack_bf16(v[2], v[3]);
    w.z = pack_bf16(v[4], v[5]);
    w.w = pack_bf16(v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) = w;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// ---------------------------------------------------------------- norm and rotation

struct NormRopeArgs {
  const void *q, *k, *qw, *kw;
  void *qo, *ko;
  const float* inv_freq;
  const int32_t* positions;
  long long q_sn, q_sh, k_sn, k_sh, qo_sn, qo_sh, ko_sn, ko_sh;
  int N, Hq, Hkv, D, R, interleaved;
  float eps;
  int hpg;     // heads a thread group takes of one token
  int groups;  // thread groups a token needs: ceil((Hq + Hkv) / hpg)
};

// The rotation by position p and frequency f is by p f / 2pi turns, of which
// only the fraction counts. f / 2pi is held as a 64-bit binary fraction F (its
// own error 2^-56 of a turn from the fp64 quotient), so p F modulo 2^64 is
// that fraction: one integer product, no 64-bit floating point per position,
// and an error below 2^-24 of a turn for positions up to 2^31.
SV_DEVINL unsigned long long turn_fraction(float inv_freq) {
  const double t = (double)inv_freq * 0.15915494309189533577;
  const double f = t - floor(t);
  const unsigned hi = __double2uint_rd(f * 4294967296.0);
  const unsigned lo = __double2uint_rd((f * 4294967296.0 - (double)hi) * 4294967296.0);
  return ((unsigned long long)hi << 32) | lo;
}

// cos and sin of the position's turn, from the top 32 bits of the fraction.
SV_DEVINL float2 turn_cos_sin(int position, unsigned long long F) {
  const unsigned long long t = F * (unsigned long long)(long long)position;
  float s, c;
  sincospif((float)(int)(t >> 32) * 4.656612873077393e-10f, &s, &c);
  return make_float2(c, s);
}

// 16 bytes as loaded (eight bf16 or four fp32 values).
template <int DT, int VEC>
SV_DEVINL void unpack(const uint4& w, float (&v)[VEC]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SV_BF16) {
      v[2 * i] = bf16_lo(x[i]);
      v[2 * i + 1] = bf16_hi(x[i]);
    } else {
      v[i] = __uint_as_float(x[i]);
    }
  }
}
template <int DT>
SV_DEVINL uint4 raw_vec(const void* base, long long at) {
  return *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + at * (DT == SV_BF16 ? 2 : 4));
}

// A thread group of L lanes takes `hpg` heads of one token, one after another with the
// next one's loads under way. Its lanes hold 2 VEC elements of a row each, as two
// 16-byte vectors: with halves, vector s and its partner R/2 further (the pair that
// rotates together, so nothing crosses lanes); interleaved, or past R, two vectors that
// each stand alone. The angles are computed once and serve the group's heads: with one
// head a group their cosines and sines bound the kernel (137 us for 16383 tokens of
// 40 heads of 128 in bf16); so it takes 67 us, 5.0 TB/s, with 72 % of the issue slots active and
// the memory 54 %: its instructions bound it now. fp32: 121 us, 5.6 TB/s.
// Blocks of 128 threads: 77 us with 256, whose last blocks are fewer and longer.
template <int DT, int L, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a) {
  constexpr int VEC = DT == SV_BF16 ? 8 : 4;
  extern __shared__ unsigned long long frac[];  // [R/2]
  for (int i = threadIdx.x; i < a.R / 2; i += kThreads) frac[i] = turn_fraction(a.inv_freq[i]);
  __syncthreads();
  const int lane = threadIdx.x % L;
  const int slots = a.D / (2 * VEC);       // lanes with work
  const int rot = a.R / (2 * VEC);         // of which the first `rot` rotate
  // Element offsets of the lane's two vectors.
  int e0, e1;
  if (INTER || lane >= rot) {
    e0 = lane * 2 * VEC;
    e1 = e0 + VEC;
  } else {
    e0 = lane * VEC;
    e1 = e0 + a.R / 2;
  }
  const bool turns = lane < rot;
  const float inv_d = 1.0f / (float)a.D;
  const long long g = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool live = lane < slots && g < (long long)a.N * a.groups;
  const int H = a.Hq + a.Hkv;
  const int n = live ? (int)(g / a.groups) : 0;
  const int h0 = live ? (int)(g % a.groups) * a.hpg : 0;
  const int h1 = live ? min(H, h0 + a.hpg) : 0;
  float cs[VEC], sn[VEC];
  if (turns && live) {
    const int pos = a.positions[n];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float2 c = turn_cos_sin(pos, frac[lane * VEC + i]);
      cs[i] = c.x;
      sn[i] = c.y;
    }
  }
  // All lanes of a warp stay in the loop (the sums are exchanged warp-wide).
  uint4 raw[2], ahead[2];
  auto fetch = [&](int h, uint4 (&to)[2]) {
    to[0] = to[1] = make_uint4(0, 0, 0, 0);
    if (h >= h1) return;
    const bool isq = h < a.Hq;
    const void* src = isq ? a.q : a.k;
    const long long at = isq ? n * a.q_sn + h * a.q_sh : n * a.k_sn + (h - a.Hq) * a.k_sh;
    to[0] = raw_vec<DT>(src, at + e0);
    to[1] = raw_vec<DT>(src, at + e1);
  };
  fetch(h0, raw);
#pragma unroll 1
  for (int i = 0; i < a.hpg; ++i) {
    const int h = h0 + i;
    fetch(h + 1, ahead);  // the next head's row while this one is worked on
    const bool on = h < h1, isq = h < a.Hq;
    float x0[VEC], x1[VEC];
    unpack<DT, VEC>(raw[0], x0);
    unpack<DT, VEC>(raw[1], x1);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (on) {
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      if (isq ? a.qw != nullptr : a.kw != nullptr) {
        float w0[VEC], w1[VEC];
        load_vec<DT, VEC>(isq ? a.qw : a.kw, e0, w0);
        load_vec<DT, VEC>(isq ? a.qw : a.kw, e1, w1);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x0[i] *= r * w0[i];
          x1[i] *= r * w1[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x0[i] *= r;
          x1[i] *= r;
        }
      }
      if (turns) {
        if (INTER) {
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const float p = x0[i], s = x0[i + 1], t = x1[i], u = x1[i + 1];
            x0[i] = p * cs[i / 2] - s * sn[i / 2];
            x0[i + 1] = s * cs[i / 2] + p * sn[i / 2];
            x1[i] = t * cs[(VEC + i) / 2] - u * sn[(VEC + i) / 2];
            x1[i + 1] = u * cs[(VEC + i) / 2] + t * sn[(VEC + i) / 2];
          }
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float p = x0[i], s = x1[i];
            x0[i] = p * cs[i] - s * sn[i];
            x1[i] = s * cs[i] + p * sn[i];
          }
        }
      }
      void* dst = isq ? a.qo : a.ko;
      const long long to = isq ? n * a.qo_sn + h * a.qo_sh : n * a.ko_sn + (h - a.Hq) * a.ko_sh;
      store_vec<DT, VEC>(dst, to + e0, x0);
      store_vec<DT, VEC>(dst, to + e1, x1);
    }
    raw[0] = ahead[0];
    raw[1] = ahead[1];
  }
}

// Any even R <= D, any D, any strides: one warp a row, element loads. The row
// is read again for the rotation (from L1) after the sum of squares; a pair's
// two elements belong to one lane, so in-place calls are sound. A block takes up to
// kAnyHeads heads of one token and computes its angles once: with fractions of a turn (fp64,
// at 1/64 of the rate) for each row, 16383 tokens of 40 heads of 100 in bf16 took 763 us, so 226 (1.2 TB/s).
constexpr int kAnyHeads = 16;
template <int DT>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(NormRopeArgs a) {
  extern __shared__ float2 turns[];  // [R/2]
  const int lane = threadIdx.x & 31;
  const int H = a.Hq + a.Hkv, groups = (H + kAnyHeads - 1) / kAnyHeads;
  const int n = (int)(blockIdx.x / (unsigned)groups), h0 = (int)(blockIdx.x % (unsigned)groups) * kAnyHeads;
  const int half = a.R / 2;
  const int pos = a.positions[n];
  for (int i = threadIdx.x; i < half; i += kThreads) turns[i] = turn_cos_sin(pos, turn_fraction(a.inv_freq[i]));
  __syncthreads();
  for (int h = h0 + (int)(threadIdx.x >> 5); h < min(H, h0 + kAnyHeads); h += kThreads / 32) {
    const bool isq = h < a.Hq;
    const void* src = isq ? a.q : a.k;
    void* dst = isq ? a.qo : a.ko;
    const void* w = isq ? a.qw : a.kw;
    const long long at = isq ? n * a.q_sn + h * a.q_sh : n * a.k_sn + (h - a.Hq) * a.k_sh;
    const long long to = isq ? n * a.qo_sn + h * a.qo_sh : n * a.ko_sn + (h - a.Hq) * a.ko_sh;
    float ss = 0.0f, v[1];
    for (int e = lane; e < a.D; e += 32) {
      load_vec<DT, 1>(src, at + e, v);
      ss = fmaf(v[0], v[0], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = 1.0f / sqrtf(fmaf(ss, 1.0f / (float)a.D, a.eps));
    for (int i = lane; i < half; i += 32) {
      const int i0 = a.interleaved ? 2 * i : i, i1 = a.interleaved ? 2 * i + 1 : i + half;
      float x0[1], x1[1], w0[1] = {1.0f}, w1[1] = {1.0f};
      load_vec<DT, 1>(src, at + i0, x0);
      load_vec<DT, 1>(src, at + i1, x1);
      if (w) {
        load_vec<DT, 1>(w, i0, w0);
        load_vec<DT, 1>(w, i1, w1);
      }
      const float2 c = turns[i];
      const float p = x0[0] * (r * w0[0]), s = x1[0] * (r * w1[0]);
      const float y0[1] = {p * c.x - s * c.y}, y1[1] = {s * c.x + p * c.y};
      store_vec<DT, 1>(dst, to + i0, y0);
      store_vec<DT, 1>(dst, to + i1, y1);
    }
    for (int e = a.R + lane; e < a.D; e += 32) {
      float x[1], ww[1] = {1.0f};
      load_vec<DT, 1>(src, at + e, x);
      if (w) load_vec<DT, 1>(w, e, ww);
      const float y[1] = {x[0] * (r * ww[0])};
      store_vec<DT, 1>(dst, to + e, y);
    }
  }
}

// ---------------------------------------------------------------- the quantised cache

struct CacheArgs {
  const void *k, *v;      // write: rows in; read: unused
  void *ko, *vo;          // read: rows out
  const long long* slots;
  void *kc, *vc;
  float *ks, *vs;
  unsigned* status;
  long long k_sn, k_sh, v_sn, v_sh;  // strides of the rows in or out
  long long num_slots;
  int N, H, D, P;
};

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxMin = 1e-30f;  // keeps 448 / amax finite

SV_DEVINL uint32_t e4m3_pair(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

SV_DEVINL float2 e4m3_unpack(uint32_t pair) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(pair & 0xffffu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// max that keeps a NaN of either operand (fmaxf drops it).
SV_DEVINL float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The row of (token n, head h): element offset in the cache and index of its
// scale. Rows of one page and head are consecutive.
SV_DEVINL long long cache_row(const CacheArgs& a, long long slot, int h) {
  const long long page = slot / a.P;
  return (page * a.H + h) * a.P + (slot - page * a.P);
}

// A slot outside the cache (other than -1, which skips the row) sets a status
// bit; the row is skipped too.
SV_DEVINL bool slot_ok(const CacheArgs& a, long long slot) {
  if (slot >= 0 && slot < a.num_slots) return true;
  if (slot != -1 && a.status) atomicOr(a.status, (unsigned)SV_DEV_SLOT_RANGE);
  return false;
}

// L lanes take HB heads of one token, key and value together, 16 elements of each row a
// lane: one slot leads to 2 HB rows whose loads are in flight together. A row's scale
// is its largest magnitude over 448, the largest e4m3 value, so that no code saturates
// but by rounding. A row with NaN or infinity gets a NaN scale and codes of zero: it
// reads back as NaN everywhere. Bound by memory: 32767 tokens of 8 heads of 128, bf16 to
// e4m3, take 33 us, 5.8 TB/s; bf16 to bf16 42 us, fp32 to e4m3 54 us. Heads a group, in blocks of 256: one 37 us, two 34, four 40.
template <int DT, int CDT, int L, int HB>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheArgs a) {
  constexpr int VEC = DT == SV_BF16 ? 8 : 4;
  constexpr int NV = 16 / VEC;
  const int lane = threadIdx.x % L;
  const int quads = (a.H + HB - 1) / HB;
  const long long item = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  const bool row = item < (long long)a.N * quads;
  const int n = row ? (int)(item / quads) : 0, h0 = row ? (int)(item % quads) * HB : 0;
  const long long slot = row ? a.slots[n] : -1;
  const bool on = row && lane * 16 < a.D && slot_ok(a, slot);
  uint4 raw[HB][2][NV];
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int h = h0 + j;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        raw[j][w][i] = make_uint4(0, 0, 0, 0);
        if (on && h < a.H)
          raw[j][w][i] = raw_vec<DT>(w ? a.v : a.k, (w ? n * a.v_sn + h * a.v_sh : n * a.k_sn + h * a.k_sh) +
                                                        lane * 16 + i * VEC);
      }
    }
  }
  const long long r0 = on ? cache_row(a, slot, h0) : 0;
#pragma unroll
  for (int j = 0; j < HB; ++j) {
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[16], amax = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float t[VEC];
        unpack<DT, VEC>(raw[j][w][i], t);
#pragma unroll
        for (int k = 0; k < VEC; ++k) x[i * VEC + k] = t[k];
      }
      if constexpr (CDT == SV_E4M3) {
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(x[i]));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      }
      if (!on || h0 + j >= a.H) continue;
      const long long r = r0 + (long long)j * a.P;
      void* c = w ? a.vc : a.kc;
      if constexpr (CDT == SV_E4M3) {
        const bool bad = !(amax < INFINITY);
        const float top = fmaxf(amax, kAmaxMin);
        const float inv = bad ? 0.0f : __fdiv_rn(kE4m3Max, top);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = bad ? 0.0f : x[4 * i + k] * inv;
          o[i] = e4m3_pair(y[0], y[1]) | (e4m3_pair(y[2], y[3]) << 16);
        }
        *reinterpret_cast<uint4*>(static_cast<unsigned char*>(c) + r * a.D + lane * 16) =
            make_uint4(o[0], o[1], o[2], o[3]);
        if (lane == 0) (w ? a.vs : a.ks)[r] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(top, kE4m3Max);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) t[k] = x[8 * i + k];
          store_vec<SV_BF16, 8>(c, r * a.D + lane * 16 + 8 * i, t);
        }
      }
    }
  }
}

// The same division; 100003 tokens of 8 heads of 128, e4m3 to bf16, take 101 us, 6.1 TB/s; bf16 to
// bf16 125 us, e4m3 to fp32 231 us (4.5 TB/s).
// Heads a group, in blocks of 256: one 105 us, two 102, four 106.
template <int DT, int CDT, int L, int HB>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheArgs a) {
  constexpr int VEC = DT == SV_BF16 ? 8 : 4;
  constexpr int NV = 16 / VEC, CV = CDT == SV_E4M3 ? 1 : 2;  // 16-byte vectors of a lane's elements
  const int lane = threadIdx.x % L;
  const int quads = (a.H + HB - 1) / HB;
  const long long item = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  if (item >= (long long)a.N * quads || lane * 16 >= a.D) return;
  const int n = (int)(item / quads), h0 = (int)(item % quads) * HB;
  const long long slot = a.slots[n];
  const bool ok = slot_ok(a, slot);
  const long long r0 = ok ? cache_row(a, slot, h0) : 0;
  uint4 raw[HB][2][CV];
  float scale[HB][2];
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const long long r = r0 + (long long)j * a.P;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const bool on = ok && h0 + j < a.H;
      scale[j][w] = 0.0f;
#pragma unroll
      for (int i = 0; i < CV; ++i) {
        raw[j][w][i] = make_uint4(0, 0, 0, 0);
        if (on)
          raw[j][w][i] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(w ? a.vc : a.kc) +
                                                         (r * a.D + lane * 16) * CV + 16 * i);
      }
      if (CDT == SV_E4M3 && on) scale[j][w] = (w ? a.vs : a.ks)[r];
    }
  }
#pragma unroll
  for (int j = 0; j < HB; ++j) {
    const int h = h0 + j;
    if (h >= a.H) break;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      float x[16];
      if constexpr (CDT == SV_E4M3) {
        const float s = scale[j][w];
        const uint32_t u[4] = {raw[j][w][0].x, raw[j][w][0].y, raw[j][w][0].z, raw[j][w][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 lo = e4m3_unpack(u[i]), hi = e4m3_unpack(u[i] >> 16);
          x[4 * i] = lo.x * s;
          x[4 * i + 1] = lo.y * s;
          x[4 * i + 2] = hi.x * s;
          x[4 * i + 3] = hi.y * s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < CV; ++i) {
          float t[8];
          unpack<SV_BF16, 8>(raw[j][w][i], t);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[8 * i + k] = t[k];
        }
      }
      const long long to = (w ? n * a.v_sn + h * a.v_sh : n * a.k_sn + h * a.k_sh) + lane * 16;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float t[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) t[k] = x[i * VEC + k];
        store_vec<DT, VEC>(w ? a.vo : a.ko, to + i * VEC, t);
      }
    }
  }
}

// Any D, any alignment: one warp a row, element accesses. 16383 tokens of 8 heads of 100, bf16
// and e4m3: written in 92 us, read in 68 (0.9 and 1.2 TB/s).
template <int DT, int CDT>
__global__ void __launch_bounds__(kThreads) cache_write_any_kernel(CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= 2ll * a.N * a.H) return;
  const int w = (int)(item & 1);
  const int n = (int)((item >> 1) / a.H), h = (int)((item >> 1) % a.H);
  const long long slot = a.slots[n];
  if (!slot_ok(a, slot)) return;
  const long long r = cache_row(a, slot, h);
  const void* src = w ? a.v : a.k;
  const long long at = w ? n * a.v_sn + h * a.v_sh : n * a.k_sn + h * a.k_sh;
  void* c = w ? a.vc : a.kc;
  float x[1];
  if constexpr (CDT == SV_E4M3) {
    float amax = 0.0f;
    for (int e = lane; e < a.D; e += 32) {
      load_vec<DT, 1>(src, at + e, x);
      amax = max_nan(amax, fabsf(x[0]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const bool bad = !(amax < INFINITY);
    const float top = fmaxf(amax, kAmaxMin);
    const float inv = bad ? 0.0f : __fdiv_rn(kE4m3Max, top);
    for (int e = lane; e < a.D; e += 32) {
      load_vec<DT, 1>(src, at + e, x);
      static_cast<unsigned char*>(c)[r * a.D + e] =
          (unsigned char)e4m3_pair(bad ? 0.0f : x[0] * inv, 0.0f);
    }
    if (lane == 0) (w ? a.vs : a.ks)[r] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(top, kE4m3Max);
  } else {
    for (int e = lane; e < a.D; e += 32) {
      load_vec<DT, 1>(src, at + e, x);
      store_vec<SV_BF16, 1>(c, r * a.D + e, x);
    }
  }
}

template <int DT, int CDT>
__global__ void __launch_bounds__(kThreads) cache_read_any_kernel(CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (item >= 2ll * a.N * a.H) return;
  const int w = (int)(item & 1);
  const int n = (int)((item >> 1) / a.H), h = (int)((item >> 1) % a.H);
  const long long slot = a.slots[n];
  const bool ok = slot_ok(a, slot);
  const long long r = ok ? cache_row(a, slot, h) : 0;
  const void* c = w ? a.vc : a.kc;
  const long long to = w ? n * a.v_sn + h * a.v_sh : n * a.k_sn + h * a.k_sh;
  for (int e = lane; e < a.D; e += 32) {
    float x[1] = {0.0f};
    if (ok) {
      if constexpr (CDT == SV_E4M3)
        x[0] = e4m3_unpack(static_cast<const unsigned char*>(c)[r * a.D + e]).x * (w ? a.vs : a.ks)[r];
      else
        load_vec<SV_BF16, 1>(c, r * a.D + e, x);
    }
    store_vec<DT, 1>(w ? a.vo : a.ko, to + e, x);
  }
}

// ---------------------------------------------------------------- host side

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

unsigned blocks_for(long long items, int per_block) {
  return (unsigned)((items + per_block - 1) / per_block);
}

// Lanes that share a row of `units` vectors: the next power of two.
int lanes_for(int units) {
  int l = 1;
  while (l < units) l <<= 1;
  return l;
}

template <int DT, int L>
void launch_norm_rope(const NormRopeArgs& a, unsigned grid, cudaStream_t st) {
  const size_t smem = (size_t)(a.R / 2) * 8;
  if (a.interleaved)
    norm_rope_kernel<DT, L, true><<<grid, kThreads, smem, st>>>(a);
  else
    norm_rope_kernel<DT, L, false><<<grid, kThreads, smem, st>>>(a);
}

template <int DT>
cudaError_t norm_rope(NormRopeArgs a, bool vec, cudaStream_t st) {
  constexpr int VEC = DT == SV_BF16 ? 8 : 4;
  const int H = a.Hq + a.Hkv;
  if (!vec) {
    norm_rope_any_kernel<DT><<<blocks_for((long long)a.N * ((H + kAnyHeads - 1) / kAnyHeads), 1), kThreads,
                               a.R / 2 * sizeof(float2), st>>>(a);
    return cudaGetLastError();
  }
  const int L = lanes_for(a.D / (2 * VEC));
  const int per_block = kThreads / L;
  // Heads a group: one where the call is small and latency counts; else as many as leave
  // eight blocks an SM, so that the angles are shared.
  a.hpg = 1;
  for (int hpg = 4; hpg <= 16; hpg *= 2)
    if (H >= hpg && (long long)a.N * ((H + hpg - 1) / hpg) >= 8ll * kSms * per_block) a.hpg = hpg;
  a.groups = (H + a.hpg - 1) / a.hpg;
  a.hpg = (H + a.groups - 1) / a.groups;  // evenly
  const unsigned grid = blocks_for((long long)a.N * a.groups, per_block);
  switch (L) {
    case 1: launch_norm_rope<DT, 1>(a, grid, st); break;
    case 2: launch_norm_rope<DT, 2>(a, grid, st); break;
    case 4: launch_norm_rope<DT, 4>(a, grid, st); break;
    case 8: launch_norm_rope<DT, 8>(a, grid, st); break;
    case 16: launch_norm_rope<DT, 16>(a, grid, st); break;
    default: launch_norm_rope<DT, 32>(a, grid, st); break;
  }
  return cudaGetLastError();
}

template <int DT, int CDT, bool READ, int L, int HB>
void launch_cache_hb(const CacheArgs& a, cudaStream_t st) {
  const unsigned grid = blocks_for((long long)a.N * ((a.H + HB - 1) / HB), kThreads / L);
  if (READ)
    cache_read_kernel<DT, CDT, L, HB><<<grid, kThreads, 0, st>>>(a);
  else
    cache_write_kernel<DT, CDT, L, HB><<<grid, kThreads, 0, st>>>(a);
}

// Two heads a group (four loads of 16 bytes and more in flight a lane) where that leaves eight
// blocks an SM; one in small calls.
template <int DT, int CDT, bool READ, int L>
void launch_cache_l(const CacheArgs& a, cudaStream_t st) {
  if (a.H >= 2 && (long long)a.N * ((a.H + 1) / 2) >= 8ll * kSms * (kThreads / L))
    launch_cache_hb<DT, CDT, READ, L, 2>(a, st);
  else
    launch_cache_hb<DT, CDT, READ, L, 1>(a, st);
}

template <int DT, int CDT, bool READ>
cudaError_t launch_cache(const CacheArgs& a, bool vec, cudaStream_t st) {
  if (!vec) {
    const unsigned grid = blocks_for(2ll * a.N * a.H, kThreads / 32);
    if (READ)
      cache_read_any_kernel<DT, CDT><<<grid, kThreads, 0, st>>>(a);
    else
      cache_write_any_kernel<DT, CDT><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
  }
  switch (lanes_for(a.D / 16)) {
    case 1: launch_cache_l<DT, CDT, READ, 1>(a, st); break;
    case 2: launch_cache_l<DT, CDT, READ, 2>(a, st); break;
    case 4: launch_cache_l<DT, CDT, READ, 4>(a, st); break;
    case 8: launch_cache_l<DT, CDT, READ, 8>(a, st); break;
    case 16: launch_cache_l<DT, CDT, READ, 16>(a, st); break;
    default: launch_cache_l<DT, CDT, READ, 32>(a, st); break;
  }
  return cudaGetLastError();
}

// The checks that cache_write and cache_read share; SV_OK with N == 0 means
// that nothing is to be done.
template <bool READ>
int run_cache(CacheArgs a, long long num_pages, int dtype, int cache_dtype, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  if (cache_dtype != SV_BF16 && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (a.N < 0 || a.H < 1 || a.H > 1024 || a.D < 1 || a.D > kHeadDimMax || a.P < 1 || num_pages < 1)
    return SV_ERR_SHAPE;
  // N * H rows fill at most 2^31 - 1 blocks; the cache stays below 2^62 elements.
  if ((long long)a.N * a.H >= (1ll << 32) || num_pages > (1ll << 31) || a.P > (1 << 20)) return SV_ERR_SHAPE;
  if (a.N == 0) return SV_OK;
  const void* rows_k = READ ? a.ko : a.k;
  const void* rows_v = READ ? a.vo : a.v;
  if (!rows_k || !rows_v || !a.slots || !a.kc || !a.vc) return SV_ERR_NULL;
  if (cache_dtype == SV_E4M3 && (!a.ks || !a.vs)) return SV_ERR_NULL;
  const size_t es = dtype == SV_BF16 ? 2 : 4, ces = cache_dtype == SV_BF16 ? 2 : 1;
  if (misaligned(rows_k, es) || misaligned(rows_v, es) || misaligned(a.slots, 8) ||
      misaligned(a.kc, ces) || misaligned(a.vc, ces) || misaligned(a.status, 4) ||
      (cache_dtype == SV_E4M3 && (misaligned(a.ks, 4) || misaligned(a.vs, 4))))
    return SV_ERR_ALIGN;
  a.num_slots = num_pages * a.P;
  const long long per16 = 16 / (long long)es;
  const bool vec = a.D % 16 == 0 && a.D <= 512 && !misaligned(rows_k, 16) && !misaligned(rows_v, 16) &&
                   !misaligned(a.kc, 16) && !misaligned(a.vc, 16) && a.k_sn % per16 == 0 &&
                   a.k_sh % per16 == 0 && a.v_sn % per16 == 0 && a.v_sh % per16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SV_BF16)
    e = cache_dtype == SV_BF16 ? launch_cache<SV_BF16, SV_BF16, READ>(a, vec, st)
                               : launch_cache<SV_BF16, SV_E4M3, READ>(a, vec, st);
  else
    e = cache_dtype == SV_BF16 ? launch_cache<SV_F32, SV_BF16, READ>(a, vec, st)
                               : launch_cache<SV_F32, SV_E4M3, READ>(a, vec, st);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace tio
}  // namespace sv

using namespace sv::tio;

extern "C" {

int sv_qk_norm_rope(const void* q, int64_t q_stride_n, int64_t q_stride_h, const void* k,
                    int64_t k_stride_n, int64_t k_stride_h, const void* q_weight,
                    const void* k_weight, const float* inv_freq, const int32_t* positions, int N,
                    int Hq, int Hkv, int D, int R, int dtype, float eps, int interleaved, void* q_out,
                    int64_t qo_stride_n, int64_t qo_stride_h, void* k_out, int64_t ko_stride_n,
                    int64_t ko_stride_h, void* stream) {
  if (dtype != SV_BF16 && dtype != SV_F32) return SV_ERR_DTYPE;
  if (N < 0 || Hq < 0 || Hkv < 0 || Hq + Hkv < 1 || Hq > 1024 || Hkv > 1024 || D < 1 ||
      D > sv::kHeadDimMax || R < 0 || R > D || R % 2 != 0 || !(eps >= 0.0f) || std::isinf(eps))
    return SV_ERR_SHAPE;
  // At most 2^31 - 1 blocks: odd sizes take kAnyHeads heads of a token a block, the others no fewer rows.
  if ((long long)N * ((Hq + Hkv + kAnyHeads - 1) / kAnyHeads) >= (1ll << 31)) return SV_ERR_SHAPE;
  if (N == 0) return SV_OK;
  if ((Hq && (!q || !q_out)) || (Hkv && (!k || !k_out)) || (R && !inv_freq) || !positions)
    return SV_ERR_NULL;
  const size_t es = dtype == SV_BF16 ? 2 : 4;
  if (misaligned(q, es) || misaligned(k, es) || misaligned(q_out, es) || misaligned(k_out, es) ||
      misaligned(q_weight, es) || misaligned(k_weight, es) || misaligned(inv_freq, 4) ||
      misaligned(positions, 4))
    return SV_ERR_ALIGN;
  NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.qw = q_weight;
  a.kw = k_weight;
  a.qo = q_out;
  a.ko = k_out;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.q_sn = q_stride_n;
  a.q_sh = q_stride_h;
  a.k_sn = k_stride_n;
  a.k_sh = k_stride_h;
  a.qo_sn = qo_stride_n;
  a.qo_sh = qo_stride_h;
  a.ko_sn = ko_stride_n;
  a.ko_sh = ko_stride_h;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.R = R;
  a.interleaved = interleaved != 0;
  a.eps = eps;
  const int per16 = (int)(16 / es);
  const int64_t strides[8] = {q_stride_n, q_stride_h, k_stride_n, k_stride_h,
                              qo_stride_n, qo_stride_h, ko_stride_n, ko_stride_h};
  bool vec = D % (2 * per16) == 0 && R % (2 * per16) == 0 && D / (2 * per16) <= 32 &&
             !misaligned(q, 16) && !misaligned(k, 16) && !misaligned(q_out, 16) &&
             !misaligned(k_out, 16) && !misaligned(q_weight, 16) && !misaligned(k_weight, 16);
  for (int64_t s : strides) vec = vec && s % per16 == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SV_BF16 ? norm_rope<SV_BF16>(a, vec, st) : norm_rope<SV_F32>(a, vec, st);
  return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int sv_cache_write(const void* k, int64_t k_stride_n, int64_t k_stride_h, const void* v,
                   int64_t v_stride_n, int64_t v_stride_h, const int64_t* slots, int N, int Hkv,
                   int D, int dtype, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                   int64_t num_pages, int page_size, int cache_dtype, uint32_t* status, void* stream) {
  CacheArgs a{};
  a.k = k;
  a.v = v;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.kc = k_cache;
  a.vc = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.status = status;
  a.k_sn = k_stride_n;
  a.k_sh = k_stride_h;
  a.v_sn = v_stride_n;
  a.v_sh = v_stride_h;
  a.N = N;
  a.H = Hkv;
  a.D = D;
  a.P = page_size;
  return run_cache<false>(a, num_pages, dtype, cache_dtype, stream);
}

int sv_cache_read(const void* k_cache, const void* v_cache, const float* k_scale,
                  const float* v_scale, int64_t num_pages, int page_size, int cache_dtype,
                  const int64_t* slots, int N, int Hkv, int D, int dtype, void* k_out,
                  int64_t ko_stride_n, int64_t ko_stride_h, void* v_out, int64_t vo_stride_n,
                  int64_t vo_stride_h, uint32_t* status, void* stream) {
  CacheArgs a{};
  a.ko = k_out;
  a.vo = v_out;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.kc = const_cast<void*>(k_cache);
  a.vc = const_cast<void*>(v_cache);
  a.ks = const_cast<float*>(k_scale);
  a.vs = const_cast<float*>(v_scale);
  a.status = status;
  a.k_sn = ko_stride_n;
  a.k_sh = ko_stride_h;
  a.v_sn = vo_stride_n;
  a.v_sh = vo_stride_h;
  a.N = N;
  a.H = Hkv;
  a.D = D;
  a.P = page_size;
  return run_cache<true>(a, num_pages, dtype, cache_dtype, stream);
}

}  // extern "C"
