// The sparse attention's kernel for few query heads a key/value head (sv_sparse_decode.cu).
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace sv {
namespace sparse {
namespace dec {

struct Args {
  const __nv_bfloat16* q;
  long long q_sn, q_sh;
  const void *kc, *vc;
  const float *ks, *vs;
  const int32_t *table, *ctx, *parent;  // of an item (row, key/value head): its pages; of a row: its last key, -1 at
                                        // fault; -2 for an empty row
  __nv_bfloat16* out;
  unsigned *status, *counters;
  float2* part_ml;  // [items splits][heads]: maximum and sum of a part
  float* part_o;    // [items splits][heads][D]
  int N, Hq, Hkv, D, P, budget, splits;
  float scale;
};

// Shapes that the kernel takes: heads of a key/value head are the N of an 8-wide product, and a
// block of 16 keys lies in one page.
inline bool takes(int heads, int D, int page_size) {
  return heads <= 8 && (D == 64 || D == 128) && page_size % 16 == 0;
}

// CTAs of an item: one wave in all (four a SM), but no fewer than 128 keys a CTA. Measured, us of a call with 608 / 912 /
// 1216 / 1824 CTAs wanted (pages not yet looked up ahead): 32 rows of 8 heads and 48 pages of 64, bf16 85 / 88 / 88 / 95, e4m3 75 / 78 / 77 / 86; 36 rows
// of 32 pages 66 / 73 / 73 / 86: what a CTA does before and after its keys costs more than uneven lengths.
inline int splits_of(long long items, int budget, int page_size) {
  const long long keys = (long long)budget * page_size;
  const long long want = 608 / (items > 0 ? items : 1);
  return (int)std::max(1ll, std::min({want, keys / 128, 64ll}));
}

// Room for parts (items times splits): the most that any number of items up to this one has, since fewer items are split
// further. A workspace for a batch then serves every smaller one.
inline long long most_parts(long long items, int budget, int page_size) {
  const long long keys = (long long)budget * page_size;
  return std::min(std::max(608ll, items), items * std::max(1ll, std::min(keys / 128, 64ll)));
}

// Enqueues the attention behind the selection, whose kernel clears the counters and the status word.
int launch(const Args& a, int cache_dtype, cudaStream_t st);

}  // namespace dec
}  // namespace sparse
}  // namespace sv
