// The plan of a step's pages (sv_page_plan): from the requests' lengths, the pages
// that each gets from a ring of free ones or gives back to it, and every packed
// token's slot, position and request.
#include <cstdint>
#include <algorithm>

#include <cuda_runtime.h>

#include "../../include/spec_verify.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace plan {

// The requests are summed over (tokens, pages wanted, pages given back) by one block, then the tokens and the
// pages are filled in: by the same block where there are few tokens, else by a grid that is launched
// beside it and waits on the device. Up to 1024 requests the blocks of the grid have all records in shared memory, so that
// a token's request costs no further trip to memory (1024 requests, 226 thousand tokens: 12.7 us on the device). Pages are taken
// from the head of the ring and given back behind its tail: what a call reads and writes
// of the ring does not overlap, and neither do the table's entries, so that no
// order within the call matters.

constexpr int kThreads = 1024;
constexpr int kOneBlockTokens = 4096;  // (a second launch costs what a block needs for a few turns)

struct Args {
  int32_t* ring;
  long long capacity;
  const int32_t* state_in;
  int32_t* state_out;
  int32_t* page_table;
  const int32_t *held, *ctx, *add;
  int32_t *held_out, *granted;
  int B, W, P;
  int max_tokens;
  int64_t* slots;
  int32_t *positions, *seqs;
  unsigned* status;
  // Workspace: the ring's head and tail, then a record a request.
  int32_t* head;
  long long* tok_end;  // packed tokens up to and with the request's
  int4* pages;         // first page's index from the head, pages taken, held, first index behind the tail (-1: none back)
};

struct Sums {
  long long tokens, pages, back;
};

SV_DEVINL Sums add3(const Sums& a, const Sums& b) { return {a.tokens + b.tokens, a.pages + b.pages, a.back + b.back}; }

SV_DEVINL Sums shfl_up3(const Sums& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.tokens, o), __shfl_up_sync(0xffffffffu, a.pages, o),
          __shfl_up_sync(0xffffffffu, a.back, o)};
}

// Records of up to 1024 requests.
struct Records {
  int tok_end[kThreads];  // packed tokens up to and with the request's, 2^31 - 1 at most
  int first[kThreads];    // a token's position is first + its place
  int4 pages[kThreads];   // as Args::pages
};

// One block: the sums over the requests and what each request gets. `short_end`, `first` and `pages` are
// where records go in the short form, else (NULL) they go to a.tok_end and a.pages.
SV_DEVINL void sum_requests(const Args& a, int* short_end, int* first, int4* pages_out, int* ht) {
  __shared__ Sums warps[kThreads / 32];
  __shared__ long long used_all;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long head = a.state_in[0], count = a.state_in[1];
  const bool ring_ok = head >= 0 && head < a.capacity && count >= 0 && count <= a.capacity;
  unsigned faults = ring_ok ? 0u : (unsigned)SV_DEV_PAGE_RANGE;
  // Pages come back only if the ring has room for all of them.
  long long back_all = 0;
  for (int b = tid; b < a.B; b += kThreads)
    if (a.add[b] == -1 && a.held[b] >= 0 && a.held[b] <= a.W) back_all += a.held[b];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) back_all += __shfl_xor_sync(0xffffffffu, back_all, o);
  if (lane == 0) warps[warp].back = back_all;
  if (tid == 0) used_all = 0;
  __syncthreads();
  back_all = 0;
#pragma unroll 1
  for (int i = 0; i < kThreads / 32; ++i) back_all += warps[i].back;
  const bool back_ok = ring_ok && count + back_all <= a.capacity;
  if (!back_ok) faults |= SV_DEV_PAGE_RANGE;

  Sums before{0, 0, 0};
  long long used = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    Sums x{0, 0, 0};
    long long add = 0, held = 0;
    bool valid = false, done = false, given = false;
    if (b < a.B) {
      add = a.add[b];
      held = a.held[b];
      const long long ctx = a.ctx[b];
      const bool held_ok = held >= 0 && held <= a.W;
      done = add == -1;
      if (done) {
        given = held_ok && back_ok;
        x.back = given ? held : 0;
        if (!held_ok) faults |= SV_DEV_PAGE_RANGE;
      } else {
        const long long wanted = (ctx + max(add, 0ll) + a.P - 1) / a.P;
        valid = add >= 0 && ctx >= 0 && held_ok && wanted <= a.W && ring_ok;
        if (!valid) faults |= SV_DEV_PAGE_RANGE;
        x.tokens = max(add, 0ll);
        x.pages = valid ? max(0ll, wanted - held) : 0;
      }
    }
    Sums s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = shfl_up3(s, o);
      if (lane >= o) s = add3(s, y);
    }
    __syncthreads();
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    Sums all{0, 0, 0}, mine{0, 0, 0};
    {
      Sums w = warps[lane];  // (32 warps)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Sums y = shfl_up3(w, o);
        if (lane >= o) w = add3(w, y);
      }
      all = {__shfl_sync(0xffffffffu, w.tokens, 31), __shfl_sync(0xffffffffu, w.pages, 31),
             __shfl_sync(0xffffffffu, w.back, 31)};
      const int from = warp > 0 ? warp - 1 : 0;
      mine = {__shfl_sync(0xffffffffu, w.tokens, from), __shfl_sync(0xffffffffu, w.pages, from),
              __shfl_sync(0xffffffffu, w.back, from)};
      if (warp == 0) mine = {0, 0, 0};
    }
    s = add3(add3(s, mine), before);
    before = add3(before, all);
    if (b < a.B) {
      const bool fits = valid && (x.pages == 0 || s.pages <= count);
      const bool room = s.tokens <= a.max_tokens;
      const bool ok = fits && room;
      if (valid && !fits) faults |= SV_DEV_NO_PAGES;
      if (valid && !room) faults |= SV_DEV_SLOT_RANGE;
      const long long take = ok ? x.pages : 0;
      used += take;
      const int4 pages = make_int4((int)(s.pages - x.pages), ok ? (int)take : -1, (int)held,
                                   x.back > 0 ? (int)(s.back - x.back) : -1);
      const int granted = done ? -1 : ok ? (int)add : 0, left = given ? 0 : (int)(held + take);
      if (short_end) {
        short_end[b] = (int)min(s.tokens, 0x7fffffffll);
        first[b] = (int)(a.ctx[b] - (s.tokens - x.tokens));
      } else {
        a.tok_end[b] = s.tokens;
      }
      pages_out[b] = pages;
      a.granted[b] = granted;
      a.held_out[b] = left;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) used += __shfl_xor_sync(0xffffffffu, used, o);
  if (lane == 0 && used) atomicAdd(reinterpret_cast<unsigned long long*>(&used_all), (unsigned long long)used);
  if (faults && a.status) atomicOr(a.status, faults);
  __syncthreads();
  if (tid == 0) {
    ht[0] = ring_ok ? (int)head : 0;
    ht[1] = ring_ok ? (int)((head + count) % a.capacity) : 0;
    a.state_out[0] = ring_ok ? (int)((head + used_all) % a.capacity) : (int)head;
    a.state_out[1] = ring_ok ? (int)(count - used_all + before.back) : (int)count;
  }
}

// Place of an index below twice the ring's size.
SV_DEVINL long long wrap(long long i, long long capacity) { return i < capacity ? i : i - capacity; }

// A warp a request: its new pages into the table, or its old ones back to the ring; eight loads under way.
SV_DEVINL void move_pages(const Args& a, const int4* pages, long long head, long long tail, int warp, int warps, int lane) {
#pragma unroll 1
  for (int b = warp; b < a.B; b += warps) {
    const int4 r = pages[b];
    int32_t* row = a.page_table + (long long)b * a.W;
    const bool back = r.w >= 0;
    const int n = back ? r.z : r.y;
    int32_t page[8];
#pragma unroll 1
    for (int i0 = lane; i0 < n; i0 += 256) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + 32 * u;
        if (i < n) page[u] = back ? row[i] : a.ring[wrap(head + r.x + i, a.capacity)];
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + 32 * u;
        if (i < n) (back ? a.ring[wrap(tail + r.w + i, a.capacity)] : row[r.z + i]) = page[u];
      }
    }
  }
}

// Tokens and pages, by block `block` of `blocks`.
SV_DEVINL void fill(const Args& a, int block, int blocks) {
  const int tid = threadIdx.x, lane = tid & 31;
  const long long head = a.head[0], tail = a.head[1];
  // A warp takes 32 consecutive tokens: the first one's request by a search 32 wide, the others from there.
  const int warps = blocks * (kThreads / 32);
#pragma unroll 1
  for (long long t0 = ((long long)block * (kThreads / 32) + (tid >> 5)) * 32; t0 < a.max_tokens; t0 += warps * 32ll) {
    int lo = 0, hi = a.B;  // the first request whose tokens end behind t0 lies in [lo, hi]
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + (lane + 1) * step, hi) - 1;
      const unsigned m = __ballot_sync(0xffffffffu, a.tok_end[at] > t0);
      if (m == 0) {
        lo = hi;
        break;
      }
      const int k = __ffs(m) - 1;
      hi = __shfl_sync(0xffffffffu, at, k);
      lo += k * step;
    }
    // The other lanes' requests: those of the next 32 whose tokens end before the lane's.
    const long long t = t0 + lane;
    int b = lo;
    for (bool more = true; more; lo += 32) {
      const int end = lo + lane < a.B ? (int)min(a.tok_end[lo + lane] - t0, 32ll) : 32;
      int before = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) before += __shfl_sync(0xffffffffu, end, i) <= lane;
      b += b == lo ? before : 0;
      more = __any_sync(0xffffffffu, before == 32);
    }
    if (t >= a.max_tokens) continue;
    long long slot = -1;
    int pos = -1, seq = -1;
    if (b < a.B) {
      const int4 r = a.pages[b];
      if (r.y >= 0) {
        seq = b;
        pos = a.ctx[b] + (int)(t - (a.tok_end[b] - a.add[b]));
        const int h = pos / a.P;
        const int page = h < r.z ? a.page_table[(long long)b * a.W + h]
                                 : a.ring[wrap(head + r.x + (h - r.z), a.capacity)];
        slot = (long long)page * a.P + pos % a.P;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.seqs[t] = seq;
  }
  move_pages(a, a.pages, head, tail, block * (kThreads / 32) + (tid >> 5), warps, lane);
}

// The same from records in the short form, in shared memory.
SV_DEVINL void fill_short(const Args& a, const Records& rec, long long head, long long tail, int block, int blocks) {
  const int tid = threadIdx.x, threads = blocks * kThreads;
  int b = 0;
#pragma unroll 1
  for (long long t = block * kThreads + tid; t < a.max_tokens; t += threads) {
    if (b >= a.B || rec.tok_end[b] <= t) {
      int hi = a.B;  // the first request from b on whose tokens end behind t
      while (b < hi) {
        const int mid = (b + hi) >> 1;
        if (rec.tok_end[mid] > t)
          hi = mid;
        else
          b = mid + 1;
      }
    }
    long long slot = -1;
    int pos = -1, seq = -1;
    if (b < a.B) {
      const int4 r = rec.pages[b];
      if (r.y >= 0) {
        seq = b;
        pos = rec.first[b] + (int)t;
        const int h = pos / a.P;
        const int page = h < r.z ? a.page_table[(long long)b * a.W + h] : a.ring[wrap(head + r.x + (h - r.z), a.capacity)];
        slot = (long long)page * a.P + (pos - h * a.P);
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.seqs[t] = seq;
  }
  move_pages(a, rec.pages, head, tail, block * (kThreads / 32) + (tid >> 5), threads / 32, tid & 31);
}

// Alone (few requests and tokens), or before a grid that fills.
__global__ void __launch_bounds__(kThreads) plan_one_kernel(const __grid_constant__ Args a) {
  __shared__ Records rec;
  __shared__ int ht[2];
  sum_requests(a, rec.tok_end, rec.first, rec.pages, ht);
  __syncthreads();
  fill_short(a, rec, ht[0], ht[1], 0, 1);
}

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ Args a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int* ends = a.B <= kThreads ? reinterpret_cast<int*>(a.tok_end) : nullptr;
  sum_requests(a, ends, ends ? ends + a.B : nullptr, a.pages, a.head);
}

__global__ void __launch_bounds__(kThreads) fill_short_kernel(const __grid_constant__ Args a) {
  __shared__ Records rec;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int* ends = reinterpret_cast<const int*>(a.tok_end);
  const long long head = a.head[0], tail = a.head[1];
  if (tid < a.B) {
    rec.tok_end[tid] = ends[tid];
    rec.first[tid] = ends[a.B + tid];
    rec.pages[tid] = a.pages[tid];
  }
  __syncthreads();
  fill_short(a, rec, head, tail, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kThreads) fill_kernel(const __grid_constant__ Args a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  fill(a, blockIdx.x, gridDim.x);
}

}  // namespace plan
}  // namespace sv

using namespace sv::plan;
using sv::misaligned;

extern "C" {

size_t sv_page_plan_workspace_size(int B) {
  if (B < 0) return 0;
  return 256 + sv::align_up((size_t)B * 8, 256) + sv::align_up((size_t)B * 16, 256);
}

int sv_page_plan(int32_t* ring, int64_t capacity, const int32_t* state, int32_t* page_table, const int32_t* held,
                 const int32_t* ctx_lens, const int32_t* new_lens, int B, int max_pages, int page_size, int max_tokens,
                 int64_t* slots, int32_t* positions, int32_t* seqs, int32_t* granted, int32_t* held_out,
                 int32_t* state_out, void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  if (B < 0 || max_pages < 1 || page_size < 1 || max_tokens < 0 || capacity < 1 || capacity >= (1ll << 31) ||
      (long long)max_pages * page_size >= (1ll << 31))
    return SV_ERR_SHAPE;
  if (!ring || !state || !state_out || !workspace || (max_tokens > 0 && (!slots || !positions || !seqs)) ||
      (B > 0 && (!page_table || !held || !ctx_lens || !new_lens || !granted || !held_out)))
    return SV_ERR_NULL;
  if (misaligned(ring, 4) || misaligned(state, 4) || misaligned(page_table, 4) || misaligned(held, 4) ||
      misaligned(ctx_lens, 4) || misaligned(new_lens, 4) || misaligned(slots, 8) || misaligned(positions, 4) ||
      misaligned(seqs, 4) || misaligned(granted, 4) || misaligned(held_out, 4) || misaligned(state_out, 4) ||
      misaligned(workspace, 256) || misaligned(status, 4))
    return SV_ERR_ALIGN;
  if (workspace_bytes < sv_page_plan_workspace_size(B)) return SV_ERR_WORKSPACE;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  Args a{};
  a.ring = ring;
  a.capacity = capacity;
  a.state_in = state;
  a.state_out = state_out;
  a.page_table = page_table;
  a.held = held;
  a.ctx = ctx_lens;
  a.add = new_lens;
  a.held_out = held_out;
  a.granted = granted;
  a.B = B;
  a.W = max_pages;
  a.P = page_size;
  a.max_tokens = max_tokens;
  a.slots = slots;
  a.positions = positions;
  a.seqs = seqs;
  a.status = status;
  a.head = reinterpret_cast<int32_t*>(ws);
  a.tok_end = reinterpret_cast<long long*>(ws + 256);
  a.pages = reinterpret_cast<int4*>(ws + 256 + sv::align_up((size_t)B * 8, 256));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (B <= kThreads && max_tokens <= kOneBlockTokens) {
    plan_one_kernel<<<1, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SV_OK : SV_ERR_CUDA;
  }
  plan_kernel<<<1, kThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  const long long need = std::max(((long long)max_tokens + kThreads - 1) / kThreads, ((long long)B + 31) / 32);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(304ll, need));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, B <= kThreads ? fill_short_kernel : fill_kernel, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // extern "C"
