// Attention of single query rows over lists of pages, for up to eight query heads a
// key/value head (the second kernel of sv_sparse_attention).
#include <cfloat>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"
#include "sv_sparse.h"

namespace sv {
namespace sparse {
namespace dec {

// An item is a query row and a key/value head; CTAs split its keys, and the last one to finish joins
// the parts. A warp takes 16 keys at a time, straight from global memory to the registers of
// m16n8k16 products, with no shared memory between:
//   - S (16 keys x 8 heads) = K q^T. The sum over channels may take them in any order, so a lane's 16-byte
//     pieces of a key are its A fragments as they are, with q's in the same order as B.
//   - O^T (channels x heads) += V^T P. A lane loads the same channels of four keys, and a byte permutation
//     makes pairs of keys of them; the rows of a tile are whatever channels the lanes hold.
//     P goes from S's layout to B's by an 8 x 8 transposition each.
// There is little to compute for what is read (24 products a block of 16 keys), so that warps with all their loads
// under way are what counts: 12 or more a SM, 8 KB each (codes: 4). A running maximum per head moves only when a score
// exceeds it by more than 2^8, so that most blocks need one vote; a row's sum stays per lane until
// the end. P enters as two values of 16 bits, with a product each, so that outputs are off by no more than their own
// rounding (one value alone: error against 64 bits 0.0019 for bf16, 0.0016 with both; 32 rows take as long in bf16, 72 us
// in place of 71 in e4m3). bf16 caches: 2^-16 of each weight. e4m3 caches: codes become fp16 (exact), q is
// fp16 relative to its largest value (2^-25 of that at most), and a weight times its value's scale is two fp16
// raised so that the largest is near fp16's largest (2^-22 of itself, or 2^-40 of the largest).
// 32 rows of 32/8 heads of 128: 72 us alone for 393 MB of bf16 (5.5 TB/s, DRAM 69 % active), 52 us for 204 MB of e4m3
// (3.9 TB/s, DRAM 50 % active, issue slots 36 %: of a warp's time 41 % waits for its loads, which are not under way while it
// converts, and 22 % for results of its own instructions). On the kernel for trees of few rows, with 128-wide products of
// which 4 columns are used, a whole call took 97 (bf16) and 94 us (e4m3), where it was 91 and 78 with this one; 36 rows
// of 64/8 heads 84 and 75, one row of 131072 keys 41 and 32.

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr float kNone = -FLT_MAX;  // no score is below (but for -inf)
constexpr float kLazy = 8.0f;
constexpr float kTiny = 1e-36f;   // products below count as 0 (the scale of a row of zeros is above)
constexpr float kRaise = 128.0f;  // products go up to 2^8 of their reference: raised to 2^15, below fp16's largest

SV_DEVINL void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
SV_DEVINL void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool F8>
SV_DEVINL void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F8)
    mma_f16(d, a, b0, b1);
  else
    mma_bf16(d, a, b0, b1);
}
// An 8 x 8 matrix of 16-bit values (row lane/4, columns 2 (lane % 4) and the next) transposed.
SV_DEVINL uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two e4m3 codes (the low or the high half of w) as fp16.
SV_DEVINL uint32_t codes_f16(uint32_t w, int half) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(half ? w >> 16 : w));
  return r;
}
SV_DEVINL uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
SV_DEVINL uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's bytes of a block of 16 keys: of keys g and g + 8 (lane = 4 g + c) every fourth 16 bytes from c on, of
// values 2c, 2c + 1, 2c + 8 and 2c + 9 the channels of group g.
template <int D, bool F8>
struct Block {
  static constexpr int ROW = F8 ? D : 2 * D;   // bytes of a row
  static constexpr int KP = ROW / 64;          // 16-byte pieces of a key
  static constexpr int VB = ROW / 8;           // bytes of a value
  static constexpr int VW = VB / 4;            // words of a value
  uint32_t k[2][KP * 4], v[4][VW];
  float ks[2], vs[2];
};

template <int D, bool F8>
SV_DEVINL void load_block(Block<D, F8>& x, const Args& a, long long row0, int left, int lane) {
  using B = Block<D, F8>;
  const int g = lane >> 2, c = lane & 3;
  const unsigned char* kb = static_cast<const unsigned char*>(a.kc) + row0 * B::ROW + c * 16;
  const unsigned char* vb = static_cast<const unsigned char*>(a.vc) + row0 * B::ROW;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int key = g + 8 * i;
#pragma unroll
    for (int p = 0; p < B::KP; ++p) {
      uint4 w = make_uint4(0, 0, 0, 0);
      if (key < left) w = ld_global_nc_v4(kb + key * B::ROW + p * 64);
      x.k[i][4 * p] = w.x, x.k[i][4 * p + 1] = w.y, x.k[i][4 * p + 2] = w.z, x.k[i][4 * p + 3] = w.w;
    }
    if constexpr (F8) {
      x.ks[i] = key < left ? __ldg(a.ks + row0 + key) : 0.0f;
      x.vs[i] = key < left ? __ldg(a.vs + row0 + key) : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = 2 * c + (i & 1) + 8 * (i >> 1);
    // Channels of group g: 16-byte pieces 128 bytes apart (bf16), or the group's bytes of the row (codes).
    if constexpr (B::VB >= 16) {
#pragma unroll
      for (int p = 0; p < B::VB / 16; ++p) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (key < left) w = ld_global_nc_v4(vb + key * B::ROW + p * 128 + g * 16);
        x.v[i][4 * p] = w.x, x.v[i][4 * p + 1] = w.y, x.v[i][4 * p + 2] = w.z, x.v[i][4 * p + 3] = w.w;
      }
    } else {
      uint2 w = make_uint2(0, 0);
      if (key < left) w = __ldg(reinterpret_cast<const uint2*>(vb + key * B::ROW + g * 8));
      x.v[i][0] = w.x, x.v[i][1] = w.y;
    }
  }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 4) sparse_decode_kernel(const __grid_constant__ Args a) {
  using B = Block<D, F8>;
  constexpr int STEPS = D / 16;
  __shared__ float so[kWarps][8][D];
  __shared__ float sm[kWarps][8], smv[kWarps][8], sl[kWarps][8];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x % a.splits;
  const long long item = blockIdx.x / a.splits, n = item / a.Hkv;
  const int h = (int)(item % a.Hkv), G = a.Hq / a.Hkv;
  // q in the order of the keys' pieces, head g's (heads beyond the group: 0); this call's own input, so before the wait.
  const __nv_bfloat16* qr = a.q + n * a.q_sn + (long long)(h * G + min(g, G - 1)) * a.q_sh;
  uint32_t q[STEPS][2];
#pragma unroll
  for (int p = 0; p < D / 32; ++p) {
    // (e4m3: 16 channels a piece of a key, two pieces of q)
    const int at = F8 ? (c + 4 * (p / 2)) * 16 + (p & 1) * 8 : (c + 4 * p) * 8;
    uint4 w = *reinterpret_cast<const uint4*>(qr + at);
    if (g >= G) w = make_uint4(0, 0, 0, 0);
    q[2 * p][0] = w.x, q[2 * p][1] = w.y, q[2 * p + 1][0] = w.z, q[2 * p + 1][1] = w.w;
  }
  float qscale[2] = {a.scale * 1.4426950408889634f, a.scale * 1.4426950408889634f};  // of heads 2c and 2c + 1
  if constexpr (F8) {
    uint32_t top2 = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) top2 = bf16x2_max(top2, bf16x2_max(q[s][0] & 0x7fff7fffu, q[s][1] & 0x7fff7fffu));
    float top = fmaxf(bf16_lo(top2), bf16_hi(top2));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // A power of two at or below the largest (fp32's least normal one for subnormals, 2^7 of which are whole; 1 for
    // infinities, which stay).
    const unsigned e = max(__float_as_uint(top) & 0x7f800000u, 0x00800000u);
    const float unit = e == 0x7f800000u ? 1.0f : __uint_as_float(e), down = __fdiv_rn(1.0f, unit);
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) q[s][i] = pack_f16(bf16_lo(q[s][i]) * down, bf16_hi(q[s][i]) * down);
    qscale[0] *= __shfl_sync(0xffffffffu, unit, 8 * c);      // lane 4 (2c)
    qscale[1] *= __shfl_sync(0xffffffffu, unit, 8 * c + 4);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ctx = __ldcg(a.ctx + n), parent = __ldcg(a.parent + n);
  if (ctx < 0 || parent == -2) {
    if (split != 0) return;
    if (ctx < 0 && tid == 0) atomicOr(a.status, (unsigned)SV_DEV_PAGE_RANGE);
    const __nv_bfloat16 fill = __float2bfloat16_rn(ctx < 0 ? __int_as_float(0x7fc00000) : 0.0f);
    for (int i = tid; i < G * D; i += kThreads) a.out[(n * a.Hq + h * G) * D + i] = fill;
    return;
  }
  const int keys = ctx + 1, blocks = (keys + 15) / 16;
  const int used = max(1, min(a.splits, blocks / 8));  // (no fewer than 128 keys a CTA)
  if (split >= used) return;
  const int b0 = (int)((long long)split * blocks / used), b1 = (int)((long long)(split + 1) * blocks / used);
  const int32_t* table = a.table + item * a.budget;
  const int per_page = a.P / 16;

  float o[D / 16][4] = {};
  float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};    // heads 2c, 2c + 1
  float ref[2] = {0.0f, 0.0f}, inv[2] = {0.0f, 0.0f};  // what a weight times its scale is relative to (e4m3)
  // The next block's page is looked up while one is worked on (32 rows of bf16 83 us with it, 86 without). One block at a
  // time: with two of e4m3 32 rows took 76 us, against 70, since their registers spill; so they do with the next
  // block's loads under way (74). Prefetching its lines to L2 was slower too (bf16 87, e4m3 73).
  auto page_of = [&](int b) { return __ldcg(table + min(b, b1 - 1) / per_page); };
  int id = page_of(b0 + warp);
#pragma unroll 1
  for (int b = b0 + warp; b < b1; b += kWarps) {
    const int left = keys - b * 16;
    B x;
    load_block<D, F8>(x, a, ((long long)id * a.Hkv + h) * a.P + (b % per_page) * 16, left, lane);
    id = page_of(b + kWarps);
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      uint32_t f[4];
      if constexpr (F8) {
        // Step t: words t and half of a word each.
        f[0] = codes_f16(x.k[0][t], 0), f[1] = codes_f16(x.k[1][t], 0);
        f[2] = codes_f16(x.k[0][t], 1), f[3] = codes_f16(x.k[1][t], 1);
      } else {
        f[0] = x.k[0][2 * t], f[1] = x.k[1][2 * t], f[2] = x.k[0][2 * t + 1], f[3] = x.k[1][2 * t + 1];
      }
      mma<F8>(s, f, q[t][0], q[t][1]);
    }
    // Scores in powers of two: s[0], s[1] of key g, s[2], s[3] of key g + 8.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[i] *= F8 ? qscale[i & 1] * x.ks[i >> 1] : qscale[i & 1];
      if (g + 8 * (i >> 1) >= left) s[i] = -INFINITY;
    }
    const bool grows = s[0] > m[0] + kLazy || s[2] > m[0] + kLazy || s[1] > m[1] + kLazy || s[3] > m[1] + kLazy;
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float t = fmaxf(m[i], fmaxf(s[i], s[i + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
        const float f = ex2_fast(m[i] - t);
        l[i] *= f;
        if constexpr (F8) {
          ref[i] *= f;  // O stays: its reference is what shrinks
          if (ref[i] < kTiny) ref[i] = 0.0f;
          inv[i] = ref[i] > 0.0f ? __fdiv_rn(kRaise, ref[i]) : 0.0f;
        } else {
#pragma unroll
          for (int t2 = 0; t2 < D / 16; ++t2) o[t2][i] *= f, o[t2][i + 2] *= f;
        }
        m[i] = t;
      }
    }
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = ex2_fast(s[i] - m[i & 1]);
      l[i & 1] += p[i];
      if constexpr (F8) p[i] *= x.vs[i >> 1];
    }
    if constexpr (F8) {
      const bool past = fmaxf(fabsf(p[0]), fabsf(p[2])) > 256.0f * ref[0] || fmaxf(fabsf(p[1]), fabsf(p[3])) > 256.0f * ref[1];
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = fmaxf(ref[i], fmaxf(fabsf(p[i]), fabsf(p[i + 2])));
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
          if (t < kTiny) t = 0.0f;
          inv[i] = t > 0.0f ? __fdiv_rn(kRaise, t) : 0.0f;
          const float f = ref[i] * inv[i] * (1.0f / kRaise);
#pragma unroll
          for (int t2 = 0; t2 < D / 16; ++t2) o[t2][i] *= f, o[t2][i + 2] *= f;
          ref[i] = t;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] *= inv[i & 1];
    }
    // A weight as two 16-bit values: its head, and what that leaves out. bf16 heads are cut off, so that the rest has
    // the weight's sign, and a weight above 0 has one above 0: an infinite value times either is the same infinity.
    float rest[4];
    uint32_t head0, head1;
    if constexpr (F8) {
      head0 = pack_f16(p[0], p[1]), head1 = pack_f16(p[2], p[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) rest[i] = p[i] - __half2float(__float2half_rn(p[i]));
    } else {
      head0 = __byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632);
      head1 = __byte_perm(__float_as_uint(p[2]), __float_as_uint(p[3]), 0x7632);
#pragma unroll
      for (int i = 0; i < 4; ++i) rest[i] = fmaxf(p[i] - bf16_hi(__float_as_uint(p[i])), fminf(p[i], 0x1p-126f));
    }
    const uint32_t p0 = transpose8(head0), p1 = transpose8(head1);
    const uint32_t rest0 = transpose8(F8 ? pack_f16(rest[0], rest[1]) : pack_bf16(rest[0], rest[1]));
    const uint32_t rest1 = transpose8(F8 ? pack_f16(rest[2], rest[3]) : pack_bf16(rest[2], rest[3]));
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = F8 ? codes_f16(x.v[i][t / 2], t & 1) : x.v[i][t];
      const uint32_t f[4] = {__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[0], w[1], 0x7632),
                             __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[2], w[3], 0x7632)};
      mma<F8>(o[t], f, p0, p1);
      mma<F8>(o[t], f, rest0, rest1);
    }
  }

  // The warps' results: channel of o[t][i]: rows g and g + 8 of tile t are channels 2 t' and 2 t' + 1 of group g.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    if (g == 0) {
      sm[warp][2 * c + i] = m[i];
      sl[warp][2 * c + i] = l[i];
      smv[warp][2 * c + i] = F8 ? ref[i] * (1.0f / kRaise) : 1.0f;
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const int ch = F8 ? g * (D / 8) + 2 * t : (t / 4) * 64 + g * 8 + 2 * (t % 4);
      so[warp][2 * c + i][ch] = o[t][i];
      so[warp][2 * c + i][ch + 1] = o[t][i + 2];
    }
  }
  __syncthreads();
  const long long part = (item * a.splits + split) * G;
  for (int i = tid; i < G * D; i += kThreads) {
    const int r = i / D, d = i % D;
    float top = kNone, sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += sl[w][r] * ex2_fast(sm[w][r] - top);
      acc += so[w][r][d] * (smv[w][r] * ex2_fast(sm[w][r] - top));  // (a warp without keys: 0)
    }
    if (used == 1) {
      a.out[(n * a.Hq + h * G) * D + i] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc / sum);
    } else {
      a.part_o[part * D + i] = acc;
      if (d == 0) a.part_ml[part + r] = make_float2(top, sum);
    }
  }
  if (used == 1) return;
  // The last CTA of the item to arrive joins the parts, in their order.
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&a.counters[item], 1u) == (unsigned)(used - 1);
  __syncthreads();
  if (!last) return;
  __threadfence();
  const long long first = item * a.splits * G;
  for (int i = tid; i < G * D; i += kThreads) {
    const int r = i / D;
    float top = kNone, sum = 0.0f, acc = 0.0f;
#pragma unroll 4
    for (int k = 0; k < used; ++k) {
      const float2 ml = __ldcg(&a.part_ml[first + k * G + r]);
      const float x = __ldcg(&a.part_o[(first + (long long)k * G) * D + i]);
      const float t = fmaxf(top, ml.x), keep = ex2_fast(top - t), f = ex2_fast(ml.x - t);
      sum = sum * keep + ml.y * f;
      acc = acc * keep + x * f;
      top = t;
    }
    a.out[(n * a.Hq + h * G) * D + i] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : acc / sum);
  }
}

template <int D, bool F8>
int launch_of(const Args& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.N * a.Hkv * a.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sparse_decode_kernel<D, F8>, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

int launch(const Args& a, int cache_dtype, cudaStream_t st) {
  if (cache_dtype == SV_E4M3) return a.D == 64 ? launch_of<64, true>(a, st) : launch_of<128, true>(a, st);
  return a.D == 64 ? launch_of<64, false>(a, st) : launch_of<128, false>(a, st);
}

}  // namespace dec
}  // namespace sparse
}  // namespace sv
