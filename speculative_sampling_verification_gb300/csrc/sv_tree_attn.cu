// Attention of a tree of drafted tokens over the paged key/value cache
// (sv_tree_attention): node i of a sequence attends the sequence's context,
// its ancestors and itself.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace tat {

constexpr int kTreeMax = 128;

struct Args {
  const __nv_bfloat16* q;
  long long q_sb, q_st, q_sh;
  const void *kc, *vc;
  const float *ks, *vs;
  const int32_t *page_table, *ctx_lens, *parents;
  __nv_bfloat16* out;
  unsigned* status;
  long long num_pages;
  int B, T, Hq, Hkv, D, P, max_pages;
  float scale;
};

// ---------------------------------------------------------------- any shape
//
// One warp a query row, one key at a time, running maximum and sum in fp32.
// Takes every head size and page size; bound by the latency of a key's
// reduction over the lanes.

constexpr int kAnyThreads = 128;
constexpr int kAnyPerLane = kHeadDimMax / 32;

template <int CDT>
SV_DEVINL float cache_elem(const void* c, long long at) {
  if constexpr (CDT == SV_E4M3) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<const unsigned char*>(c)[at], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  } else {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(c)[at]);
  }
}

template <int CDT>
__global__ void __launch_bounds__(kAnyThreads) tree_attn_any_kernel(Args a) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kAnyThreads / 32) + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.T * a.Hq) return;
  const int h = (int)(row % a.Hq);
  const int t = (int)(row / a.Hq % a.T);
  const int b = (int)(row / a.Hq / a.T);
  const int hk = h / (a.Hq / a.Hkv);
  __nv_bfloat16* out = a.out + row * a.D;

  // The tree: every node's parent is -1, an earlier node that is not padding,
  // or -2 for padding. `live` counts up to the last node that is not padding.
  const int32_t* par = a.parents ? a.parents + (long long)b * a.T : nullptr;
  bool bad_tree = false;
  int live = 0;
  for (int i = lane; i < a.T; i += 32) {
    const int p = par ? par[i] : i - 1;
    if (p < -2 || p >= i || (p >= 0 && par && par[p] == -2)) bad_tree = true;
    if (p != -2) live = i + 1;
  }
  bad_tree = __any_sync(0xffffffffu, bad_tree);
  live = __reduce_max_sync(0xffffffffu, live);
  const int ctx = a.ctx_lens[b];
  const int32_t* table = a.page_table + (long long)b * a.max_pages;
  bool bad_page = ctx < 0 || (long long)ctx + live > (long long)a.max_pages * a.P;
  if (!bad_page && !bad_tree) {
    const int need = (ctx + live + a.P - 1) / a.P;
    for (int i = lane; i < need; i += 32) {
      bool used = i * (long long)a.P < ctx;
      for (int j = max(0, i * a.P - ctx); j < live && !used && j < (i + 1) * a.P - ctx; ++j)
        used = !par || par[j] != -2;
      if (used && (table[i] < 0 || table[i] >= a.num_pages)) bad_page = true;
    }
    bad_page = __any_sync(0xffffffffu, bad_page);
  }
  if (bad_tree || bad_page) {
    if (lane == 0)
      atomicOr(a.status, (bad_tree ? (unsigned)SV_DEV_TREE : 0u) |
                             (bad_page ? (unsigned)SV_DEV_PAGE_RANGE : 0u));
    for (int e = lane; e < a.D; e += 32) out[e] = __float2bfloat16_rn(__int_as_float(0x7fc00000));
    return;
  }
  unsigned anc[kTreeMax / 32] = {};
  for (int j = t; j >= 0;) {
    const int p = par ? par[j] : j - 1;
    if (p == -2) break;
#pragma unroll
    for (int w = 0; w < kTreeMax / 32; ++w)
      if (w == j / 32) anc[w] |= 1u << (j % 32);
    j = p;
  }
  const bool dead = (par && par[t] == -2);

  float q[kAnyPerLane], acc[kAnyPerLane];
  const __nv_bfloat16* qr = a.q + b * a.q_sb + t * a.q_st + h * a.q_sh;
#pragma unroll
  for (int i = 0; i < kAnyPerLane; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < a.D ? __bfloat162float(qr[e]) : 0.0f;
    acc[i] = 0.0f;
  }
  float m = -INFINITY, sum = 0.0f;
  const int end = dead ? 0 : ctx + t + 1;
  for (int pos = 0; pos < end; ++pos) {
    if (pos >= ctx) {
      const int j = pos - ctx;
      unsigned w = 0;
#pragma unroll
      for (int i = 0; i < kTreeMax / 32; ++i)
        if (i == j / 32) w = anc[i];
      if (!(w >> (j % 32) & 1u)) continue;
    }
    const long long r = ((long long)table[pos / a.P] * a.Hkv + hk) * a.P + pos % a.P;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kAnyPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < a.D) s = fmaf(q[i], cache_elem<CDT>(a.kc, r * a.D + e), s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    s *= a.scale;
    float vs = 1.0f;
    if constexpr (CDT == SV_E4M3) {
      s *= a.ks[r];
      vs = a.vs[r];
    }
    if (!(s > -INFINITY) && !isnan(s)) continue;  // a score of -inf weighs nothing
    const float nm = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.0f : __expf(m - nm), p = __expf(s - nm);
    sum = fmaf(sum, keep, p);
    m = nm;
#pragma unroll
    for (int i = 0; i < kAnyPerLane; ++i) {
      const int e = lane + 32 * i;
      if (e < a.D) acc[i] = fmaf(acc[i], keep, p * vs * cache_elem<CDT>(a.vc, r * a.D + e));
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < kAnyPerLane; ++i) {
    const int e = lane + 32 * i;
    if (e < a.D) out[e] = __float2bfloat16_rn(acc[i] * inv);
  }
}

// ---------------------------------------------------------------- host side

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

bool sizes_ok(int B, int T, int Hq, int Hkv, int D, int max_pages, int page_size) {
  if (B < 0 || T < 1 || T > kTreeMax || Hkv < 1 || Hq < 1 || Hq > 1024 || Hq % Hkv != 0 || D < 1 ||
      D > kHeadDimMax || max_pages < 1 || page_size < 1)
    return false;
  // Positions are 32-bit, and so are the rows of a call.
  return (long long)max_pages * page_size < (1ll << 31) - kTreeMax && (long long)B * T * Hq < (1ll << 31) &&
         (long long)B * max_pages < (1ll << 40);
}

}  // namespace tat
}  // namespace sv

using namespace sv::tat;

extern "C" {

size_t sv_tree_attention_workspace_size(int B, int T, int Hq, int Hkv, int D, int max_pages,
                                        int page_size) {
  if (!sizes_ok(B, T, Hq, Hkv, D, max_pages, page_size)) return 0;
  return 256;
}

int sv_tree_attention(const void* q, int64_t q_stride_b, int64_t q_stride_t, int64_t q_stride_h,
                      const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, int64_t num_pages, int page_size, int cache_dtype,
                      const int32_t* page_table, const int32_t* ctx_lens, const int32_t* parents,
                      int B, int T, int Hq, int Hkv, int D, int max_pages, float scale, void* out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (cache_dtype != SV_BF16 && cache_dtype != SV_E4M3) return SV_ERR_DTYPE;
  if (!sizes_ok(B, T, Hq, Hkv, D, max_pages, page_size) || num_pages < 1 || num_pages > (1ll << 31) ||
      !std::isfinite(scale))
    return SV_ERR_SHAPE;
  if (B == 0) return SV_OK;
  if (!q || !k_cache || !v_cache || !page_table || !ctx_lens || !out || !workspace) return SV_ERR_NULL;
  if (cache_dtype == SV_E4M3 && (!k_scale || !v_scale)) return SV_ERR_NULL;
  const size_t ces = cache_dtype == SV_BF16 ? 2 : 1;
  if (misaligned(q, 2) || misaligned(out, 2) || misaligned(k_cache, ces) || misaligned(v_cache, ces) ||
      misaligned(page_table, 4) || misaligned(ctx_lens, 4) || misaligned(parents, 4) ||
      misaligned(workspace, 256) ||
      (cache_dtype == SV_E4M3 && (misaligned(k_scale, 4) || misaligned(v_scale, 4))))
    return SV_ERR_ALIGN;
  if (workspace_bytes < sv_tree_attention_workspace_size(B, T, Hq, Hkv, D, max_pages, page_size))
    return SV_ERR_WORKSPACE;
  Args a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_sb = q_stride_b;
  a.q_st = q_stride_t;
  a.q_sh = q_stride_h;
  a.kc = k_cache;
  a.vc = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.page_table = page_table;
  a.ctx_lens = ctx_lens;
  a.parents = parents;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.status = static_cast<unsigned*>(workspace);
  a.num_pages = num_pages;
  a.B = B;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.P = page_size;
  a.max_pages = max_pages;
  a.scale = scale;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, 4, st) != cudaSuccess) return SV_ERR_CUDA;
  const long long rows = (long long)B * T * Hq;
  const unsigned grid = (unsigned)((rows + kAnyThreads / 32 - 1) / (kAnyThreads / 32));
  if (cache_dtype == SV_E4M3)
    tree_attn_any_kernel<SV_E4M3><<<grid, kAnyThreads, 0, st>>>(a);
  else
    tree_attn_any_kernel<SV_BF16><<<grid, kAnyThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
