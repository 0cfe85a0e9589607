// The attention kernels' arguments and launch (sv_tree_attn.cu), shared with the
// sparse attention, which attends a page table of its own for every head.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

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
  int table_heads;  // rows of the page table a sequence: 1, or one for each key/value head
  int chained;      // the kernel launched just before writes page_table, ctx_lens and parents
  float scale;
};

// First entry of the pages of sequence b for key/value head hk.
__device__ __forceinline__ long long table_row(const Args& a, int b, int hk) {
  return (a.table_heads == 1 ? (long long)b : (long long)b * a.table_heads + hk) * a.max_pages;
}

bool sizes_ok(int B, int T, int Hq, int Hkv, int D, int max_pages, int page_size);

// Workspace words that must be 0 when the kernels of these sizes start; 1 for sizes
// whose kernel needs the status word alone.
size_t cleared_words(int T, int Hq, int Hkv, int D, int page_size);

// Enqueues the attention. The workspace's words are cleared here, unless a.chained:
// then the kernel before has cleared them.
int launch_attention(const Args& a, int cache_dtype, void* workspace, cudaStream_t st);

}  // namespace tat
}  // namespace sv
