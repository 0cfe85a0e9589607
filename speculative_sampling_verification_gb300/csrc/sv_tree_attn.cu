// Attention of a tree of drafted tokens over the paged key/value cache
// (sv_tree_attention): node i of a sequence attends the sequence's context,
// its ancestors and itself.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <algorithm>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

// ---------------------------------------------------------------- tensor cores
//
// Rows are (node, query head of the group) pairs that share a key/value head: a
// Q tile is up to 128 of them, the M of one tcgen05.mma. Keys come in tiles of
// KT positions. For a tile: S = Q K^T into tensor memory; two threads a row turn
// S into P = 2^(S c - m c) (c = scale log2 e) with its running maximum m and sum,
// and writes P as bf16 over S; O += P V with P as the tensor-memory operand.
// O is rescaled in tensor memory only when the maximum grows by more than 2^8
// in P (P stays below 2^8, and the result does not depend on the reference). P is
// rounded to bf16 (half a step, 2^-8) because the tensor cores take it so; the
// sums are those of the unrounded values.
//
// Two streams, each with its S, O and a warpgroup for the softmax, keep the
// tensor cores busy while a softmax runs. With at most 128 rows a key/value
// head (SHARED = false) the streams take alternate tiles of the same rows, and
// their results are joined at the end; with more rows (SHARED) each stream has a Q
// tile of its own and both use every tile. Head sizes above 128 have room for
// one stream only.
//
// 8 sequences of 64 nodes, 64/8 heads of 128, contexts to 32768, bf16: 341 us, 1.00 PFLOP/s, with
// the tensor pipe active 41 % of the time and the issue slots 38 %: the chain of product,
// softmax and product bounds it. One thread a row: 381 us. 64 sequences of 9 nodes, 32/8 heads,
// to 8192, bf16: 208 us, 5.8 TB/s. From an e4m3 cache four warps convert every code, which
// bounds it whatever the rows: 11 nodes (44 rows) 411 us, 32 nodes 437 us.
//
// Work: the tiles of all (sequence, key/value head) items, with a few units for the item
// itself before them, form one line, cut into equal ranges, one for each group of CTAs (the CTAs of a group take the item's
// Q tiles, in step, so that a tile is read from HBM once). The cuts follow the
// lengths on the device, so ragged batches and few long sequences balance
// alike. An item that lies in one range is written at once; the parts of a cut
// one go to the workspace as (O, m, sum), and the last CTA to arrive joins them in
// the order of the ranges, so that results do not depend on the timing.
//
// Warps: 0-15 softmax (a stream has eight: four for the lanes of its 128 rows, for each
// half of a tile's keys; one stream only: 0-7), 16 producer (TMA, one box a page), 17 MMA
// issuer and owner of the tensor memory, 20-23 (e4m3 cache) convert codes to bf16 between
// a staging ring and the operand ring; the scales of keys enter S, those of values
// enter P, in fp32. The softmax warps meet at hardware barriers, so none of them
// leaves early: once a wait has run out they only count their tiles down.

constexpr int kConvWarps = 4;
constexpr int kProducer = 16, kIssuer = 17, kConverter = 20;
constexpr int kMaxCtas = 152;
constexpr int kScaleSlots = 8;
constexpr int kMaxSlots = 8;
constexpr int kFewRows = 40;    // most rows of the kernel whose products have keys as their M
constexpr float kLazy = 8.0f;   // growth of the maximum (powers of two) before O is rescaled

struct TcArgs {
  Args a;
  int rows, rpt;        // rows a key/value head (T G); rows of a Q tile
  int parts_per_item;   // CTAs of a group: Q tiles (or pairs of them) of an item
  int groups;           // ranges of the line of tiles
  int box;              // keys of one TMA box: min(page, KT)
  int lp;               // log2 of the page size (a power of two here)
  float c;              // |scale| log2 e, or 1 for a scale of 0
  float join_c;         // powers of two in a unit of the parts' m
  unsigned qflip;       // sign bits to flip in Q (a negative scale)
  int qzero;            // a scale of 0: Q counts as 0
  unsigned* counters;   // [groups parts_per_item]: parts that have arrived
  float* part_o;        // [groups parts_per_item 2][rows of a CTA][D]
  float2* part_ml;      // [groups parts_per_item 2][rows of a CTA]
};

template <int DP, bool F8, bool SHARED>
struct Cfg {
  static constexpr int KT = DP == 256 ? 64 : 128;
  static constexpr int NS = DP == 256 ? 1 : 2;
  static constexpr int NQ = SHARED ? 2 : 1;
  static constexpr int kQBytes = 128 * DP * 2;
  static constexpr int kSlot = KT * DP * 2;
  static constexpr int kStage = KT * DP;
  static constexpr int kBudget = 214 * 1024;
  static constexpr int kStages = F8 ? 4 : 0;
  static constexpr int kFit = (kBudget - NQ * kQBytes - kStages * kStage - (F8 ? kScaleSlots * 2 * KT * 4 : 0)) / kSlot;
  static constexpr int kSlots = kFit < 8 ? kFit : 8;
  static constexpr bool kAlternate = NS == 2 && !SHARED;
  static constexpr int kThreads = 32 * (F8 ? kConverter + kConvWarps : kIssuer + 1);
  static constexpr unsigned kS0 = 0, kS1 = 128, kO0 = NS == 2 ? 256 : 128, kO1 = 256 + DP;
};

struct TcTail {
  unsigned long long full[kMaxSlots], empty[kMaxSlots];
  unsigned long long sfull[4], sempty[4];
  unsigned long long scale[kScaleSlots];
  unsigned long long q_ready, s_ready[2], p_ready[2], pv_done[2];
  unsigned tmem_base, abort, bad[2], badv[2], last;
  int b0;
  long long lo, hi, base0, total;
  int groups;
  int par[2][2][kTreeMax];
};

struct WideTail {
  TcTail t;
  float2 ml[2][2][128];  // [stream][half of the keys][row]: maximum and sum
  float rmax[2][2][128];
};

template <int DP, bool F8, bool SHARED>
constexpr int tc_smem() {
  using C = Cfg<DP, F8, SHARED>;
  return 1024 + C::NQ * C::kQBytes + C::kSlots * C::kSlot + C::kStages * C::kStage +
         (F8 ? kScaleSlots * 2 * C::KT * 4 : 0) + (int)sizeof(WideTail);
}

SV_DEVINL void bar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

SV_DEVINL bool bar_wait(unsigned bar, unsigned parity, volatile unsigned* abort, unsigned* status) {
  if (mbar_test_parity(bar, parity)) return true;
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (unsigned i = 0;; ++i) {
    if (mbar_test_parity(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        atomicOr(status, (unsigned)SV_DEV_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
  }
}

// The same by a whole warp, with one answer.
SV_DEVINL bool warp_wait(unsigned bar, unsigned parity, volatile unsigned* abort, unsigned* status) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, abort, status));
}

SV_DEVINL void tma_4d(unsigned dst, const CUtensorMap* map, int x, int y, int z, int w, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Descriptors of shared-memory operands in 128-byte swizzle atoms (8 rows of 128
// bytes): rows of 64 values along K (Q and K), or rows of 64 values along N (V,
// whose rows are the K of its product; `lead` bytes to the next 64 of N).
SV_DEVINL uint64_t desc_k(unsigned addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
SV_DEVINL uint64_t desc_n(unsigned addr, unsigned lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16, fp32 accumulator, bf16 operands, M = 128; B along N when `nmajor`.
SV_DEVINL uint32_t idesc(int n, bool nmajor) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((nmajor ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         (8u << 24);
}

// The whole issuing warp runs these; `lead` is nonzero in the one lane that issues.
// The operands are the same in every lane, and kept so for the compiler (uni), so
// that they stay in uniform registers: issued from a branch of one lane, each
// instruction took about 130 cycles.
SV_DEVINL unsigned elect_lane() {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
SV_DEVINL unsigned uni(unsigned v) { return __shfl_sync(0xffffffffu, v, 0); }
SV_DEVINL void mma_ss(unsigned lead, unsigned d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((unsigned)acc), "r"(lead)
      : "memory");
}
SV_DEVINL void mma_ts(unsigned lead, unsigned d, unsigned a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((unsigned)acc), "r"(lead)
      : "memory");
}
SV_DEVINL void mma_f8(unsigned lead, unsigned d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((unsigned)acc), "r"(lead)
      : "memory");
}
SV_DEVINL void commit(unsigned lead, unsigned bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
SV_DEVINL void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
SV_DEVINL void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
SV_DEVINL void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of this thread's lane.
SV_DEVINL void tmem_ld32(unsigned t, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
SV_DEVINL void tmem_ld8(unsigned t, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(t));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
SV_DEVINL void tmem_st16(unsigned t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
SV_DEVINL void tmem_ld24(unsigned t, float* v) {
  uint32_t r[24];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%24];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%25];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]),
        "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]),
        "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]),
        "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23])
      : "r"(t), "r"(t + 16));
#pragma unroll
  for (int i = 0; i < 24; ++i) v[i] = __uint_as_float(r[i]);
}
SV_DEVINL void tmem_ld4(unsigned t, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(t));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
SV_DEVINL void tmem_st4(unsigned t, float a, float b, float c, float d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(t), "f"(a), "f"(b), "f"(c),
               "f"(d)
               : "memory");
}
// Single columns: t and t + step; or three of each, `piece` apart.
SV_DEVINL void tmem_ld_1x2(unsigned t, unsigned step, float* a, float* b) {
  uint32_t r[2];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%2];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%3];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1])
      : "r"(t), "r"(t + step));
  *a = __uint_as_float(r[0]);
  *b = __uint_as_float(r[1]);
}
SV_DEVINL void tmem_ld_3x2(unsigned t, unsigned piece, unsigned step, float (&v)[6]) {
  uint32_t r[6];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%6];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%7];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%2}, [%8];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%3}, [%9];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%4}, [%10];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%5}, [%11];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5])
      : "r"(t), "r"(t + piece), "r"(t + 2 * piece), "r"(t + step), "r"(t + step + piece), "r"(t + step + 2 * piece));
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = __uint_as_float(r[i]);
}

SV_DEVINL uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
SV_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The kernel launched before this one (which cleared the counters) is complete.
SV_DEVINL void wait_for_clear() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Hardware barrier of `threads` threads, and the OR of their predicates.
SV_DEVINL void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
SV_DEVINL bool named_any(int id, int threads, bool v) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((unsigned)v), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Tiles of a sequence; a context outside its page table counts as one tile.
SV_DEVINL bool ctx_ok(const Args& a, int ctx) { return ctx >= 0 && (long long)ctx <= (long long)a.max_pages * a.P; }
template <int KT>
SV_DEVINL int tiles_of(const Args& a, int ctx) {
  return ctx_ok(a, ctx) ? (int)(((long long)ctx + a.T + KT - 1) / KT) : 1;
}

// Units of an item on the line before its tiles: what an item costs a CTA beside
// its tiles (Q, the first references, the output), in tiles. 64 sequences of 9 nodes,
// ragged to 8192 (bf16 / e4m3 cache): 6 units 219 / 218 us, 10 units 208 / 206, 14 units
// 211 / 210.
constexpr int kItemUnits = 10;

// A CTA's way along its range: the item (b, hk), its tile count, context and the
// tiles [t0, t1) of it that lie in the range.
template <int KT>
struct Walk {
  int b, hk, n, ctx, t0, t1;
  long long base, hi;  // the line's index of the item's first unit, of the range's end
  SV_DEVINL void start(const Args& a, const TcTail& t) {
    t0 = t1 = 0;
    hi = t.hi;
    if (t.lo >= hi) return;
    b = t.b0;
    ctx = a.ctx_lens[b];
    n = tiles_of<KT>(a, ctx);
    const unsigned long long rem = t.lo - t.base0;
    hk = (int)(rem / (unsigned)(n + kItemUnits));
    base = t.base0 + (long long)hk * (n + kItemUnits);
    t0 = (int)max(0ll, t.lo - base - kItemUnits);
    t1 = (int)min((long long)n, hi - base - kItemUnits);
    if (t0 >= t1) next(a);  // only units before the item's tiles
  }
  SV_DEVINL bool more() const { return t0 < t1; }
  SV_DEVINL void next(const Args& a) {
    base += n + kItemUnits;
    t0 = t1 = 0;
    if (base + kItemUnits >= hi) return;
    if (++hk == a.Hkv) {
      hk = 0;
      ctx = a.ctx_lens[++b];
      n = tiles_of<KT>(a, ctx);
    }
    t1 = (int)min((long long)n, hi - base - kItemUnits);
  }
};

// One warp: the range of tiles that is group `group`'s, from the lengths.
template <int KT>
SV_DEVINL void find_range(const TcArgs& x, TcTail& t, int group, int lane) {
  const Args& a = x.a;
  long long total = 0;
#pragma unroll 1
  for (int b = lane; b < a.B; b += 32)
    total += (long long)(tiles_of<KT>(a, a.ctx_lens[b]) + kItemUnits) * a.Hkv;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int groups = (int)min((long long)x.groups, total);
  const long long lo = group < groups ? (long long)group * total / groups : 0;
  const long long hi = group < groups ? (long long)(group + 1) * total / groups : 0;
  long long before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const long long n =
        b0 + lane < a.B ? (long long)(tiles_of<KT>(a, a.ctx_lens[b0 + lane]) + kItemUnits) * a.Hkv : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool mine = lo >= before + incl - n && lo < before + incl;
    if (mine) {
      t.b0 = b0 + lane;
      t.base0 = before + incl - n;
    }
    if (__any_sync(0xffffffffu, mine)) break;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    t.lo = lo;
    t.hi = hi;
    t.total = total;
    t.groups = groups;
  }
}

// Called by `threads` threads once their part of an item that is cut is written:
// the last part to arrive joins them all, in the order of the ranges. `sum` and O of
// a part are relative to its m (in units of 1/join_c powers of two); NaN marks a sequence at fault.
// Out of line: it runs once an item, and the kernels' code is long as it is.
template <int KT>
__device__ __noinline__ void join_parts(const TcArgs& x, TcTail& t, const Walk<KT>& w, int part, int cta_rows,
                                        int rows_here, int threads) {
  const Args& a = x.a;
  const long long total = t.total;
  const int ng = t.groups, G = a.Hq / a.Hkv;
  const long long first = w.base + kItemUnits;  // the item's first tile on the line
  const int gs = (int)(((first + 1) * ng - 1) / total), ge = (int)(((first + w.n) * ng - 1) / total);
  __threadfence();
  named_sync(3, threads);
  if (threadIdx.x == 0)
    t.last = atomicAdd(&x.counters[gs * x.parts_per_item + part], 1u) == (unsigned)(ge - gs);
  named_sync(3, threads);
  if (!t.last) return;
  __threadfence();
  const int units = a.D / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < rows_here * units; i += threads) {
    const int r = i / units, u = i - r * units;
    const int gr = part * cta_rows + r;
    if (gr >= x.rows) continue;
    // Eight parts at a time, their loads together; a running reference over the batches.
    float top = -INFINITY, l = 0.0f;
    bool poison = false;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int g0 = gs; g0 <= ge; g0 += 8) {
      float2 ml[8];
      float4 o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int g = min(g0 + k, ge);
        const long long sl = (long long)(g * x.parts_per_item + part) * 2 + (g == gs ? 1 : 0);
        ml[k] = __ldcg(&x.part_ml[sl * cta_rows + r]);
        o[k] = __ldcg(reinterpret_cast<const float4*>(x.part_o + (sl * cta_rows + r) * a.D) + u);
      }
      float nt = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (g0 + k > ge) ml[k].x = -INFINITY;
        poison = poison || isnan(ml[k].x);
        nt = fmaxf(nt, ml[k].x);
      }
      const float keep = top == -INFINITY ? 0.0f : ex2_fast((top - nt) * x.join_c);
      l *= keep;
      acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
      top = nt;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        // (A part of NaN scores alone has the maximum -inf too: its sum, NaN, still counts.)
        const float f = ml[k].x == -INFINITY ? 0.0f : ex2_fast((ml[k].x - top) * x.join_c);
        l = fmaf(ml[k].y, f, l);
        acc.x = fmaf(o[k].x, f, acc.x);
        acc.y = fmaf(o[k].y, f, acc.y);
        acc.z = fmaf(o[k].z, f, acc.z);
        acc.w = fmaf(o[k].w, f, acc.w);
      }
    }
    const int nd = gr / G;
    const bool gone = a.parents && a.parents[(long long)w.b * a.T + nd] == -2;
    float inv_l = l == 0.0f || gone ? 0.0f : 1.0f / l;
    if (poison) inv_l = __int_as_float(0x7fc00000);
    if (inv_l == 0.0f) acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(acc.x * inv_l, acc.y * inv_l);
    const __nv_bfloat162 h1 = __floats2bfloat162_rn(acc.z * inv_l, acc.w * inv_l);
    uint2 o;
    o.x = *reinterpret_cast<const uint32_t*>(&h0);
    o.y = *reinterpret_cast<const uint32_t*>(&h1);
    *reinterpret_cast<uint2*>(a.out + (((long long)w.b * a.T + nd) * a.Hq + w.hk * G + gr % G) * a.D + u * 4) = o;
  }
}

// Place of tile i's keys and values in the order of the operand ring.
template <bool ALT>
SV_DEVINL unsigned k_entry(int i) { return ALT ? (i == 0 ? 0u : 2u * i - 1u) : 2u * i; }
template <bool ALT>
SV_DEVINL unsigned v_entry(int i, int n) { return ALT ? (i == n - 1 ? 2u * n - 1u : 2u * i + 2u) : 2u * i + 1u; }

// Two e4m3 codes in the high bytes of the halves of x -> bf16 pair: the code's
// exponent and mantissa moved into bf16's place are its value times 2^-120
// (subnormals too), which the product undoes exactly. (0x7f, NaN, reads as 480:
// rows with NaN carry it in their scale.)
SV_DEVINL uint32_t e4m3_to_bf16(uint32_t x) {
  const uint32_t y = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x7b807b80u));
  return r;
}

template <int DP, bool F8, bool SHARED>
__global__ void __launch_bounds__(Cfg<DP, F8, SHARED>::kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ TcArgs x) {
  using C = Cfg<DP, F8, SHARED>;
  constexpr int KT = C::KT, NS = C::NS;
  constexpr bool ALT = C::kAlternate;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  unsigned char* ring = smem + C::NQ * C::kQBytes;
  unsigned char* stage = ring + C::kSlots * C::kSlot;
  float* scales = reinterpret_cast<float*>(stage + C::kStages * C::kStage);  // [kScaleSlots][2][KT]
  WideTail& wide = *reinterpret_cast<WideTail*>(reinterpret_cast<unsigned char*>(scales) +
                                                (F8 ? kScaleSlots * 2 * KT * 4 : 0));
  TcTail& t = wide.t;
  const Args& a = x.a;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int group = blockIdx.x / x.parts_per_item, part = blockIdx.x % x.parts_per_item;
  constexpr int kSoft = NS * 8;  // softmax warps at work

  if (warp == 0) {
    find_range<KT>(x, t, group, lane);
  } else if (warp == kProducer && lane == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&t.full[i]), F8 ? kConvWarps : 1);
      mbar_init(smem_u32(&t.empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&t.sfull[i]), 1);
      mbar_init(smem_u32(&t.sempty[i]), kConvWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) mbar_init(smem_u32(&t.scale[i]), 1);
    mbar_init(smem_u32(&t.q_ready), kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&t.s_ready[i]), 1);
      mbar_init(smem_u32(&t.p_ready[i]), 8);
      mbar_init(smem_u32(&t.pv_done[i]), 1);
    }

    t.abort = 0;
    t.bad[0] = t.bad[1] = t.badv[0] = t.badv[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&t.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_for_clear();
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = t.tmem_base;
  volatile unsigned* abort = &t.abort;
  Walk<KT> w;
  w.start(a, t);

  if (warp == kProducer) {
    // ---- TMA: entry by entry, a lane a page
    unsigned entry = 0, tile_no = 0;
    bool ok = true;
#pragma unroll 1
    for (; w.more() && ok; w.next(a)) {
      const int n = w.t1 - w.t0;
      int live = a.T;  // nodes up to the last that is not padding
      if (a.parents && (long long)w.t1 * KT > w.ctx) {
        live = 0;
        for (int i = lane; i < a.T; i += 32)
          if (a.parents[(long long)w.b * a.T + i] != -2) live = i + 1;
        live = __reduce_max_sync(0xffffffffu, live);
      }
      const bool seq_ok = ctx_ok(a, w.ctx);
#pragma unroll 1
      for (int e = 0; e < 2 * n && ok; ++e, ++entry) {
        bool isv;
        int i;
        if (ALT) {
          isv = e == 2 * n - 1 || (e >= 2 && (e & 1) == 0);
          i = isv ? (e == 2 * n - 1 ? n - 1 : e / 2 - 1) : (e + 1) / 2;
        } else {
          isv = e & 1;
          i = e >> 1;
        }
        const int tile = w.t0 + i;
        const int boxes = KT / x.box;
        const int pos = tile * KT + lane * x.box;
        int page = -1;
        if (seq_ok && lane < boxes && pos < w.ctx + live && (pos >> x.lp) < a.max_pages)
          page = a.page_table[(long long)w.b * a.max_pages + (pos >> x.lp)];
        if (page < 0 || page >= a.num_pages) page = -1;
        const unsigned hit = __ballot_sync(0xffffffffu, page >= 0);
        const int y = pos & (a.P - 1);
        unsigned bar;
        unsigned char* dst;
        unsigned limit_ok;
        if (F8) {
          const int s = (int)(entry % 4);
          limit_ok = entry < 4 || bar_wait(smem_u32(&t.sempty[s]), ((entry / 4) & 1) ^ 1, abort, a.status);
          bar = smem_u32(&t.sfull[s]);
          dst = stage + s * C::kStage;
        } else {
          const int s = (int)(entry % C::kSlots);
          limit_ok = entry < (unsigned)C::kSlots ||
                     bar_wait(smem_u32(&t.empty[s]), ((entry / C::kSlots) & 1) ^ 1, abort, a.status);
          bar = smem_u32(&t.full[s]);
          dst = ring + s * C::kSlot;
        }
        ok = __all_sync(0xffffffffu, limit_ok);
        if (!ok) break;
        const unsigned sbar = smem_u32(&t.scale[tile_no % kScaleSlots]);
        if (lane == 0) {
          // The TMA box counts whole: columns past D arrive as zeros.
          mbar_arrive_expect_tx(bar, (unsigned)__popc(hit) * x.box * DP * (F8 ? 1 : 2));
          if (F8 && !isv) mbar_arrive_expect_tx(sbar, (unsigned)__popc(hit) * x.box * 4 * 2);
        }
        __syncwarp();
        if (page >= 0) {
          const CUtensorMap* map = isv ? &map_v : &map_k;
          if (F8) {
            tma_4d(smem_u32(dst) + lane * x.box * DP, map, 0, y, w.hk, page, bar);
            if (!isv) {
              float* sc = scales + (tile_no % kScaleSlots) * 2 * KT + lane * x.box;
              const long long r = ((long long)page * a.Hkv + w.hk) * a.P + y;
              bulk_copy_g2s(smem_u32(sc), a.ks + r, x.box * 4, sbar);
              bulk_copy_g2s(smem_u32(sc + KT), a.vs + r, x.box * 4, sbar);
            }
          } else {
#pragma unroll
            for (int k = 0; k < DP / 64; ++k)
              tma_4d(smem_u32(dst) + k * KT * 128 + lane * x.box * 128, map, k * 64, y, w.hk, page, bar);
          }
        }
        if (!isv) ++tile_no;
      }
    }
    if (*abort) {  // copies in flight must land before the shared memory goes
      for (int i = 0; i < (F8 ? 4 : C::kSlots); ++i) {
        const unsigned held = F8 ? 4u : (unsigned)C::kSlots;
        if (entry < (unsigned)i + 1) break;
        const unsigned e = entry - 1 - i;
        const unsigned bar = F8 ? smem_u32(&t.sfull[e % held]) : smem_u32(&t.full[e % held]);
        const uint64_t t0 = global_ns();
        while (!mbar_test_parity(bar, (e / held) & 1) && global_ns() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == kIssuer) {
    // ---- MMA
    {
      const unsigned lead = elect_lane();
      const uint32_t id_qk = idesc(KT, false), id_pv = idesc(a.D, true);
      const int ksteps = a.D / 16;
      unsigned entry0 = 0, item = 0;
      unsigned pcount[2] = {0, 0};   // P's awaited, by stream
      bool ok = true;
      auto full = [&](unsigned e) {
        ok = ok && warp_wait(smem_u32(&t.full[e % C::kSlots]), (e / C::kSlots) & 1, abort, a.status);
        if (ok) fence_after();
        return ok;
      };
      auto qk = [&](int s, unsigned e) {
        // S of this stream holds the last P until its product is complete.
        if (pcount[s] > 0)
          ok = ok && warp_wait(smem_u32(&t.pv_done[s]), (pcount[s] - 1) & 1, abort, a.status);
        if (!ok) return;
        fence_after();
        const uint64_t q = desc_k(uni(smem_u32(smem + (SHARED ? s * C::kQBytes : 0))));
        const uint64_t k = desc_k(uni(smem_u32(ring + (e % C::kSlots) * C::kSlot)));
        const unsigned d = uni(tmem + (s ? C::kS1 : C::kS0));
#pragma unroll
        for (int i = 0; i < DP / 16; ++i)
          if (i < ksteps)
            mma_ss(lead, d, q + (((i >> 2) * 128 * 128 + (i & 3) * 32) >> 4),
                   k + (((i >> 2) * KT * 128 + (i & 3) * 32) >> 4), id_qk, i > 0);
      };
      auto pv = [&](int s, unsigned e, bool acc) {
        const uint64_t v = desc_n(uni(smem_u32(ring + (e % C::kSlots) * C::kSlot)), KT * 128);
        const unsigned p = uni(tmem + (s ? C::kS1 : C::kS0)), d = uni(tmem + (s ? C::kO1 : C::kO0));
#pragma unroll
        for (int i = 0; i < KT / 16; ++i)
          // P lies over the first half of each half of S's columns.
          mma_ts(lead, d, p + i / (KT / 32) * (KT / 2) + i % (KT / 32) * 8, v + ((i * 2048) >> 4), id_pv, acc || i > 0);
      };
      auto p_wait = [&](int s) {
        ok = ok && warp_wait(smem_u32(&t.p_ready[s]), pcount[s] & 1, abort, a.status);
        if (ok) fence_after();
        ++pcount[s];
        return ok;
      };
      auto release = [&](unsigned e) { commit(lead, smem_u32(&t.empty[e % C::kSlots])); };
#pragma unroll 1
      for (; w.more() && ok; w.next(a), ++item) {
        const int n = w.t1 - w.t0;
        ok = ok && warp_wait(smem_u32(&t.q_ready), item & 1, abort, a.status);
        if (!ok) break;
        fence_after();
        if (ALT) {
#pragma unroll 1
          for (int i = 0; i < 2 && i < n; ++i) {
            const unsigned e = entry0 + k_entry<true>(i);
            if (!full(e)) break;
            qk(i, e);
            if (!ok) break;
            release(e);
            commit(lead, smem_u32(&t.s_ready[i]));
          }
#pragma unroll 1
          for (int i = 0; i < n && ok; ++i) {
            const int s = i & 1;
            const unsigned ev = entry0 + v_entry<true>(i, n);
            if (!full(ev) || !p_wait(s)) break;
            pv(s, ev, i >= 2);
            release(ev);
            commit(lead, smem_u32(&t.pv_done[s]));
            if (i + 2 < n) {
              const unsigned e = entry0 + k_entry<true>(i + 2);
              if (!full(e)) break;
              qk(s, e);
              if (!ok) break;
              release(e);
              commit(lead, smem_u32(&t.s_ready[s]));
            }
          }
        } else {
#pragma unroll 1
          for (int i = -1; i < n && ok; ++i) {
#pragma unroll 1
            for (int s = 0; s < NS && ok; ++s) {
              if (i >= 0) {
                const unsigned ev = entry0 + 2u * i + 1u;
                if (!full(ev) || !p_wait(s)) break;
                pv(s, ev, i > 0);
                if (s == NS - 1) release(ev);
                commit(lead, smem_u32(&t.pv_done[s]));
              }
              if (i + 1 < n) {
                const unsigned e = entry0 + 2u * (i + 1);
                if (!full(e)) break;
                qk(s, e);
                if (!ok) break;
                if (s == NS - 1) release(e);
                commit(lead, smem_u32(&t.s_ready[s]));
              }
            }
          }
        }
        entry0 += 2u * n;
      }
    }
  } else if (warp < kSoft) {
    // ---- softmax, two threads a row: a half of the tile's keys each
    const int s = warp >> 3, hf = warp >> 2 & 1, q = warp & 3;  // stream, half, 32 rows
    const int wt = threadIdx.x & 127;  // row of the Q tile, and key row of V
    const int st = threadIdx.x & 255;  // thread of the stream
    constexpr int HC = KT / 2;         // keys of a half
    const unsigned lanes = (unsigned)(q * 32) << 16;
    const unsigned sbase = tmem + (s ? C::kS1 : C::kS0) + lanes + hf * HC;
    const unsigned obase = tmem + (s ? C::kO1 : C::kO0) + lanes;
    const int G = a.Hq / a.Hkv;
    const int tile_rows = x.rpt;
    const int row0 = (SHARED ? part * 2 + s : part) * tile_rows;  // first row of this thread's Q tile
    const int nrows = max(0, min(tile_rows, x.rows - row0));
    const int row = row0 + wt;
    const bool have = wt < nrows;
    const bool busy = q * 32 < nrows;  // the warp has rows
    const int node = have ? row / G : 0;
    const float c = x.c, grow = kLazy / c;
    unsigned item = 0, tile_no = 0, scount = 0, entry0 = 0;
    auto wait = [&](unsigned long long* bar, unsigned parity) { bar_wait(smem_u32(bar), parity, abort, a.status); };
#pragma unroll 1
    for (; w.more(); w.next(a), ++item) {
      const int n = w.t1 - w.t0;
      const bool seq_ok = ctx_ok(a, w.ctx);
      const bool tail = seq_ok && (long long)w.t1 * KT > w.ctx;
      // Q into shared memory, 16 bytes a thread and step.
      {
        const int units = a.D / 8;
        constexpr int kLoaders = SHARED ? 256 : NS * 256;
        unsigned char* qs = smem + (SHARED ? s * C::kQBytes : 0);
#pragma unroll 1
        for (int i = SHARED ? st : threadIdx.x; i < 128 * units; i += kLoaders) {
          const int r = i / units, u = i - r * units;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (r < nrows && !x.qzero) {
            const int qr = row0 + r;
            v = *reinterpret_cast<const uint4*>(a.q + w.b * a.q_sb + (long long)(qr / G) * a.q_st +
                                                (long long)(w.hk * G + qr % G) * a.q_sh + u * 8);
            v.x ^= x.qflip;
            v.y ^= x.qflip;
            v.z ^= x.qflip;
            v.w ^= x.qflip;
          }
          *reinterpret_cast<uint4*>(qs + (u >> 3) * 16384 + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = v;
        }
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&t.q_ready));
      }
      // The tree and the pages, while the first keys are on their way.
      unsigned anc[4] = {};
      int* par = t.par[item & 1][s];
      {
        unsigned bad = seq_ok ? 0u : (unsigned)SV_DEV_PAGE_RANGE;
        if (tail) {
          if (st < a.T) par[st] = a.parents ? a.parents[(long long)w.b * a.T + st] : st - 1;
          named_sync(1 + s, 256);
          if (st < a.T) {
            const int p = par[st];
            if (p < -2 || p >= st || (p >= 0 && par[p] == -2)) bad |= SV_DEV_TREE;
          }
          if (have) {
#pragma unroll 1
            for (int j = node, left = a.T; j >= 0 && left > 0; --left) {
              const int p = par[j];
              if (p == -2) break;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k == j >> 5) anc[k] |= 1u << (j & 31);
              j = p < j ? p : -1;
            }
          }
        }
        if (seq_ok && s == 0) {
          const int p0 = (int)(((long long)w.t0 * KT) >> x.lp);
          const int p1 = (int)min(((long long)w.t1 * KT + a.P - 1) >> x.lp, ((long long)w.ctx + a.T + a.P - 1) >> x.lp);
#pragma unroll 1
          for (int p = p0 + st; p < p1; p += 256) {
            bool used = (long long)p * a.P < w.ctx;
            if (!used) {
              const int j1 = min((long long)a.T, (long long)(p + 1) * a.P - w.ctx);
#pragma unroll 1
              for (int j = max(0, p * a.P - w.ctx); j < j1 && !used; ++j) used = par[j] != -2;
            }
            if (!used) continue;
            const int id = p < a.max_pages ? a.page_table[(long long)w.b * a.max_pages + p] : -1;
            if (id < 0 || id >= a.num_pages) bad |= SV_DEV_PAGE_RANGE;
          }
        }
        if (bad) {
          atomicOr(&t.bad[item & 1], 1u);
          atomicOr(a.status, bad);
        }
      }

      float m = -INFINITY, sum = 0.0f;
      bool any = false;  // this stream has tiles of the item
#pragma unroll 1
      for (int i = ALT ? s : 0; i < n; i += ALT ? 2 : 1) {
        const int tile = w.t0 + i;
        const bool edge = (long long)(tile + 1) * KT > w.ctx || !seq_ok;
        const float* ksc = scales + ((tile_no + i) % kScaleSlots) * 2 * KT + hf * HC;
        wait(&t.s_ready[s], scount & 1);
        if (F8) wait(&t.scale[(tile_no + i) % kScaleSlots], ((tile_no + i) / kScaleSlots) & 1);
        fence_after();
        // Which of 32 of the half's columns from `col` on the row attends: context, then
        // ancestors; nothing in a sequence at fault.
        auto seen = [&](int col) -> unsigned {
          if (!seq_ok) return 0u;
          const long long n0 = (long long)tile * KT + hf * HC + col - w.ctx;
          if (n0 <= -32) return 0xffffffffu;
          if (n0 >= kTreeMax) return 0u;
          const int k = (int)(n0 >> 5), sh = (int)(n0 & 31);
          const unsigned lo = k < 0 ? 0xffffffffu : k == 0 ? anc[0] : k == 1 ? anc[1] : k == 2 ? anc[2] : anc[3];
          const unsigned hi = k < 0 ? anc[0] : k == 0 ? anc[1] : k == 1 ? anc[2] : k == 2 ? anc[3] : 0u;
          return __funnelshift_r(lo, hi, sh);
        };
        // S, 32 columns at a time, with the keys' scales and the mask.
        float v[32];
        auto load = [&](int col) {
          tmem_ld32(sbase + col, v);
          if (F8) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 f = *reinterpret_cast<const float4*>(ksc + col + j);
              const float2 z0 = f2_mul(make_float2(v[j], v[j + 1]), make_float2(f.x, f.y));
              const float2 z1 = f2_mul(make_float2(v[j + 2], v[j + 3]), make_float2(f.z, f.w));
              v[j] = z0.x;
              v[j + 1] = z0.y;
              v[j + 2] = z1.x;
              v[j + 3] = z1.y;
            }
          }
          if (edge) {
            const unsigned see = seen(col);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = see >> j & 1u ? v[j] : -INFINITY;
          }
        };
        float top = -INFINITY;
        if (busy) {
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int col = 0; col < HC; col += 32) {
            load(col);
#pragma unroll
            for (int j = 0; j < 32; ++j) top4[j & 3] = fmaxf(top4[j & 3], v[j]);
          }
          top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        }
        // Both threads of a row hold the same reference m: where one of the stream's rows
        // outgrows it, all take their maxima over both halves.
        if (named_any(1 + s, 256, top > m + grow || (m == -INFINITY && top > m))) {
          wide.rmax[s][hf][wt] = top;
          named_sync(1 + s, 256);
          const float nm = fmaxf(m, fmaxf(top, wide.rmax[s][hf ^ 1][wt]));
          const float f = m == -INFINITY ? 0.0f : ex2_fast((m - nm) * c);  // (1 where the row did not grow)
          if (any && busy) {
            wait(&t.pv_done[s], (scount - 1) & 1);
            fence_after();
#pragma unroll 1
            for (int col = 16 * hf; col < a.D; col += 32) {
              float v0[8], v1[8];
              uint32_t r[16];
              tmem_ld8(obase + col, v0);
              tmem_ld8(obase + col + 8, v1);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                r[j] = __float_as_uint(v0[j] * f);
                r[j + 8] = __float_as_uint(v1[j] * f);
              }
              tmem_st16(obase + col, r);
            }
          }
          sum *= f;
          m = nm;
        }
        if (busy) {
          // A masked score is -inf, so its weight comes out as 0 (the values' scales
          // may be NaN there, hence the select after them).
          const float2 c2 = f2(c), mc2 = f2(m == -INFINITY ? 0.0f : -m * c);
          float2 sum2[2] = {f2(0.0f), f2(0.0f)};
#pragma unroll
          for (int col = 0; col < HC; col += 32) {
            if (HC > 32) load(col);
            uint32_t r[16];
            const unsigned see = F8 && edge ? seen(col) : 0xffffffffu;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 y = f2_fma(make_float2(v[j], v[j + 1]), c2, mc2);
              float2 p = make_float2(ex2_fast(y.x), ex2_fast(y.y));
              sum2[(j >> 1) & 1] = f2_add(sum2[(j >> 1) & 1], p);
              if (F8) {
                p = f2_mul(p, *reinterpret_cast<const float2*>(ksc + KT + col + j));
                if (edge) {
                  p.x = see >> j & 1u ? p.x : 0.0f;
                  p.y = see >> (j + 1) & 1u ? p.y : 0.0f;
                }
              }
              r[j >> 1] = pack_bf16(p.x, p.y);
            }
            tmem_st16(sbase + col / 2, r);
          }
          const float2 sum1 = f2_add(sum2[0], sum2[1]);
          sum += sum1.x + sum1.y;
          tmem_wait_st();
        }
        // Values that no row, or not every row, may use: 0 times what lies there
        // must be 0. Dead rows are zeroed; a node's NaN or infinity is taken out
        // and given to its descendants at the end.
        if (!F8 && edge && (!SHARED || s == 0)) {
          const unsigned ev = entry0 + v_entry<ALT>(i, n);
          wait(&t.full[ev % C::kSlots], (ev / C::kSlots) & 1);
          const long long nd = (long long)tile * KT + wt - w.ctx;
          if (wt < KT && (nd >= 0 || !seq_ok)) {
            unsigned char* vrow = ring + (ev % C::kSlots) * C::kSlot + wt * 128;
            const bool dead = !seq_ok || nd >= a.T || par[nd] == -2;
#pragma unroll 1
            for (int u = hf * (DP / 16); u < (hf + 1) * (DP / 16); ++u) {
              uint4* at = reinterpret_cast<uint4*>(vrow + (u >> 3) * KT * 128 + (((u & 7) ^ (wt & 7)) << 4));
              uint4 v = dead ? make_uint4(0, 0, 0, 0) : *at;
              uint32_t z[4] = {v.x, v.y, v.z, v.w};
              bool found = dead;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if ((z[j] & 0x7f80u) == 0x7f80u) z[j] &= 0xffff0000u, found = true, t.badv[item & 1] = 1;
                if ((z[j] & 0x7f800000u) == 0x7f800000u) z[j] &= 0x0000ffffu, found = true, t.badv[item & 1] = 1;
              }
              if (found) *at = make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
          fence_async();
        }
        any = true;
        ++scount;
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&t.p_ready[s]));
      }
      tile_no += n;
      entry0 += 2u * n;

      // ---- the item's end: the streams' results joined, written or stored as a part
      if (any) wait(&t.pv_done[s], (scount - 1) & 1);
      // (A stream without tiles waits for none, so that the last item's figures may still be read:
      // it writes nothing, and nobody reads its place.)
      if (any) wide.ml[s][hf][wt] = make_float2(m, sum);
      // The next item's flags are cleared here: it sets them after the barrier, and the last
      // item's, in the same place, have been read (this item's first S, for which thread 0
      // has waited, came after every warp's arrival at q_ready).
      if (threadIdx.x == 0) t.bad[(item + 1) & 1] = t.badv[(item + 1) & 1] = 0;
      fence_before();
      named_sync(3, 32 * kSoft);
      fence_after();
      const bool bad = t.bad[item & 1] != 0;
      const bool badv = t.badv[item & 1] != 0;
      float f0 = 1.0f, f1 = 0.0f;
      if (ALT) {
        const bool two = n > 1;
        const float m0 = wide.ml[0][0][wt].x, m1 = two ? wide.ml[1][0][wt].x : -INFINITY;
        m = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.0f : ex2_fast((m0 - m) * c);
        f1 = m1 == -INFINITY ? 0.0f : ex2_fast((m1 - m) * c);
        sum = (wide.ml[0][0][wt].y + wide.ml[0][1][wt].y) * f0;
        if (two) sum += (wide.ml[1][0][wt].y + wide.ml[1][1][wt].y) * f1;
      } else {
        sum = wide.ml[s][0][wt].y + wide.ml[s][1][wt].y;
      }
      if (bad) m = __int_as_float(0x7fc00000);
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      // Eight columns a step, the row's threads in turn.
      const int col0 = 8 * (ALT ? 2 * s + hf : hf), step = ALT ? 32 : 16;
      const int cta_rows = SHARED ? 2 * tile_rows : tile_rows;
      const int prow = SHARED ? s * tile_rows + wt : wt;
      const long long slot = ((long long)(group * x.parts_per_item + part) * 2 + (w.t0 == 0 ? 1 : 0));
      float* po = x.part_o + (slot * cta_rows + prow) * a.D;
      const bool dead = have && a.parents && a.parents[(long long)w.b * a.T + node] == -2;
      const float inv = bad ? m : sum == 0.0f || dead ? 0.0f : 1.0f / sum;
      __nv_bfloat16* out = a.out + (((long long)w.b * a.T + node) * a.Hq + w.hk * G + row % G) * a.D;
      if (busy) {
#pragma unroll 1
        for (int col = col0; col < a.D; col += step) {
          __syncwarp();  // tensor memory is read by whole warps
          float v[8];
          tmem_ld8(tmem + lanes + C::kO0 + (SHARED && s ? DP : 0) + col, v);
          if (ALT) {
            float u[8];
            tmem_ld8(tmem + lanes + C::kO1 + col, u);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = v[j] * f0 + (n > 1 ? u[j] * f1 : 0.0f);
          }
          if (badv && have) {  // NaN and infinities of the nodes this row attends
#pragma unroll 1
            for (int nd = 0; nd < a.T; ++nd) {
              const long long pos = (long long)w.ctx + nd;
              if (pos < (long long)w.t0 * KT || pos >= (long long)w.t1 * KT) continue;
              unsigned word = anc[0];
#pragma unroll
              for (int k = 1; k < 4; ++k)
                if (k == nd >> 5) word = anc[k];
              if (!(word >> (nd & 31) & 1u) || (pos >> x.lp) >= a.max_pages) continue;
              const int id = a.page_table[(long long)w.b * a.max_pages + (pos >> x.lp)];
              if (id < 0 || id >= a.num_pages) continue;
              const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(a.vc) +
                                        (((long long)id * a.Hkv + w.hk) * a.P + (pos & (a.P - 1))) * a.D + col;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float y = __bfloat162float(vr[j]);
                if (!isfinite(y)) v[j] += y;
              }
            }
          }
          if (!have) continue;
          if (whole) {
            uint4 o;
            uint32_t r[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 h = __floats2bfloat162_rn(inv == 0.0f ? 0.0f : v[2 * j] * inv,
                                                             inv == 0.0f ? 0.0f : v[2 * j + 1] * inv);
              r[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            o = make_uint4(r[0], r[1], r[2], r[3]);
            *reinterpret_cast<uint4*>(out + col) = o;
          } else {
            *reinterpret_cast<float4*>(po + col) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(po + col + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        if (!whole && have && hf == 0 && (!ALT || s == 0)) x.part_ml[slot * cta_rows + prow] = make_float2(m, sum);
      }
      if (!whole) join_parts(x, t, w, part, cta_rows, SHARED ? cta_rows : nrows, 32 * kSoft);
    }
  } else if (F8 && warp >= kConverter) {
    // ---- codes to bf16: 16 of a row a thread and step
    const int ct = threadIdx.x - 32 * kConverter;
    unsigned entry = 0;
    bool ok = true;
#pragma unroll 1
    for (; w.more() && ok; w.next(a)) {
      const int n = w.t1 - w.t0;
#pragma unroll 1
      for (int e = 0; e < 2 * n && ok; ++e, ++entry) {
        const int st = (int)(entry % 4), sl = (int)(entry % C::kSlots);
        ok = bar_wait(smem_u32(&t.sfull[st]), (entry / 4) & 1, abort, a.status);
        if (ok && entry >= (unsigned)C::kSlots)
          ok = bar_wait(smem_u32(&t.empty[sl]), ((entry / C::kSlots) & 1) ^ 1, abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned char* src = stage + st * C::kStage;
        unsigned char* dst = ring + sl * C::kSlot;
        constexpr int kUnits = DP / 16;
#pragma unroll 4
        for (int i = ct; i < KT * kUnits; i += 32 * kConvWarps) {
          const int r = i / kUnits, u = i % kUnits;
          const uint4 v = *reinterpret_cast<const uint4*>(src + i * 16);
          const uint32_t z[4] = {v.x, v.y, v.z, v.w};
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[2 * j] = e4m3_to_bf16(__byte_perm(z[j], 0, 0x1404));
            o[2 * j + 1] = e4m3_to_bf16(__byte_perm(z[j], 0, 0x3424));
          }
          unsigned char* base = dst + (u >> 2) * KT * 128 + r * 128;
          const int u0 = (u & 3) * 2;
          const bool odd = (u >> 2) & 1;  // odd blocks write their halves the other way round: no bank conflicts
          const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
          *reinterpret_cast<uint4*>(base + (((u0 + odd) ^ (r & 7)) << 4)) = odd ? hi : lo;
          *reinterpret_cast<uint4*>(base + (((u0 + !odd) ^ (r & 7)) << 4)) = odd ? lo : hi;
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(smem_u32(&t.full[sl]));
          bar_arrive(smem_u32(&t.sempty[st]));
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------- tensor cores, few rows
//
// Few rows a key/value head (ordinary decoding, small trees; keys_as_m below has the
// rule): the operands change places. S^T = K Q^T has the tile's 128 keys as the M of the product and the
// rows as its N, so the tensor cores and the softmax work on the rows that exist.
// One thread a key holds that key's scores of all rows, its scales and its
// mask; the maximum of a row is not needed, only a reference m that no score (e4m3: no
// score with its value's scale, s + log2 v) exceeds by more than 2^8 (e4m3: 2^4): a vote of the
// stream's threads finds the rare tile that does, and only then are maxima taken across the
// threads and O rescaled. P^T goes to shared memory as the other operand of O^T = V^T P^T
// (M = 128 channels of the head). A row's sum is kept by each thread for its keys and joined at the item's end.
//
// An e4m3 cache feeds the tensor cores as it is (kind::f8f6f4), with no pass to
// convert it: Q and P enter as sums of e4m3 pieces. Q, scaled by a power of two to
// (224, 448], is hi + lo, exact for elements above 2^-10 of the row's largest and off by
// 2^-19 of that at most below; both multiply into the same columns. A key's part of O is its
// weight times its value's scale; P is that, relative to the reference, times 2^4, as
// p1 + p2/32 + p3/1024 with columns of O for each piece: off by at most 2^-11 of itself (a
// half's rounding) or, for small parts, 2^-24 of the reference. The reference is the row's largest
// part, not its largest weight: with a reference for the weights and one for the scales,
// one row of large values that weighed nothing drove every other part below what three
// pieces hold. The sums are relative to the same reference: 2^(s - m) stays in range for
// scales of 2^-108 (the least that sv_cache_write stores) to 2^100. A bf16 cache uses bf16
// operands, P rounded once (2^-8).
//
// 64 sequences of 9 nodes, 32/8 heads of 128, contexts to 8192, e4m3: 205 us, 3.1 TB/s, with
// 54 % of the issue slots active, the tensor pipe 13 % and the memory 40 %. With one node (4
// rows) it is 159 us: a tile's chain of product, vote, weights and product; the other 32
// rows' weights and pieces take the rest. One token over 32768 keys: 30 us, bf16 37 us.
//
// Streams, ranges and parts are those of the kernel above; the next tile's
// S^T is issued before this tile's O^T, so neither waits for the other. The softmax
// warps meet at hardware barriers, so none of them leaves early: once a wait
// has run out they only count their tiles down.

// The rows of a tile are shared by two warps for each 32 keys, RP/2 each ("halves").
template <int RP, bool F8>
struct FewCfg {
  static constexpr int KT = 128;
  static constexpr int HR = RP / 2;                                // rows of a half
  static constexpr int HS = (HR + 7) / 8 * 8;                      // its columns of S^T
  static constexpr int HN = F8 ? (3 * HR + 15) / 16 * 16 : HS;     // its columns of O^T and P
  static constexpr int N1 = 2 * HS, N2 = 2 * HN;
  static constexpr int kQBytes = N1 * 128 * 2;                     // two blocks: channels (bf16) or pieces
  static constexpr int kPBytes = KT * 128;
  static constexpr int kSlot = KT * (F8 ? 128 : 256);
  static constexpr int kTailBytes = 12 * 1024;
  static constexpr int kFit = (226 * 1024 - kTailBytes - kQBytes - 4 * kPBytes) / kSlot;
  // More in flight on each SM only lengthens the queue at the memory: an e4m3 cache's
  // batch took 217 us with every slot that fitted (at most eight), 214 with seven, 210 with five.
  static constexpr int kSlots = kFit < 6 ? kFit : 6;
  static constexpr int kSoft = 16;                                 // softmax warps
  static constexpr int kThreads = 32 * (kSoft + 2);
  static constexpr unsigned kS = 0, kO = 256;  // tensor memory: two of each, 128 columns apart
  static constexpr float kGrow = F8 ? 4.0f : 8.0f;
  static constexpr float kLift = F8 ? 16.0f : 1.0f;
};

constexpr float kNoScore = -1e30f;  // reference of a row that has seen no key
// Values' scales below 2^-100 (an unwritten slot's 0, NaN) count as this in the references, so
// that the sums of weights stay finite.
constexpr float kLeastScale = 7.888609052210118e-31f;

template <int RP>
struct FewTail {
  TcTail t;
  unsigned long long anc[2][2][64];  // [item parity][stream][node]: ancestors and itself
  unsigned long long o_done;         // the item's products are complete
  unsigned long long o_read;         // every softmax warp has read the item's O
  // Arrays that are read four values at a time lie on 16-byte boundaries.
  alignas(16) float mref[2][RP];     // [stream] references, powers of two
  alignas(16) float fac[2][RP];      // [stream] factors of a rescaling
  alignas(16) float qc[2][RP];       // [item parity] c over the row's scale of Q
  float4 fin[RP];
  float wmax[2][4][RP], wsum[2][4][RP];
  int row_out[RP];                   // a row's place in a token block of the output: node Hq + head of the group
};

template <int RP, bool F8>
constexpr int few_smem() {
  using C = FewCfg<RP, F8>;
  static_assert(sizeof(FewTail<RP>) <= C::kTailBytes, "tail");
  static_assert(C::HR % 4 == 0 && C::kQBytes % 2048 == 0, "rows of four values, blocks of 1024 bytes");
  return 1024 + C::kQBytes + 4 * C::kPBytes + C::kSlots * C::kSlot + (int)sizeof(FewTail<RP>);
}

SV_DEVINL uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Two e4m3 codes of a half pair, and the pair they stand for.
SV_DEVINL uint32_t half2_to_e4m3(__half2 h) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(half2_bits(h)));
  return r;
}
SV_DEVINL __half2 e4m3_to_half2(uint32_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)c));
  return *reinterpret_cast<const __half2*>(&r);
}

template <int N>
SV_DEVINL void tmem_ld_cols(unsigned t, float* v) {
  static_assert(N == 24 || N == 8, "columns of a half");
  if constexpr (N == 24) {
    tmem_ld24(t, v);
  } else {
    float u[8];
    tmem_ld8(t, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u[i];
  }
}

// Sums (or maxima) of v[0 .. N) over a warp: each step halves the lanes that share a row
// and the rows that a lane holds (N shuffles in all, not 5 N), in the same order every time.
template <bool MAX, int N, int O>
SV_DEVINL void halve(const float (&v)[N], int lane, int base, int count, float* out) {
  if constexpr (O == 0) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < count) out[base + j] = v[j];
  } else {
    constexpr int H = (N + 1) / 2;
    const bool up = lane & O;
    float k[H];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const float hi = j + H < N ? v[j + H] : 0.0f;
      const float mine = up ? hi : v[j], other = __shfl_xor_sync(0xffffffffu, up ? v[j] : hi, O);
      k[j] = MAX ? fmaxf(mine, other) : mine + other;
    }
    halve<MAX, H, O / 2>(k, lane, up ? base + H : base, up ? count - H : min(count, H), out);
  }
}
// Place in the operand ring: K0 K1 K2 V0 K3 V1 ... (S^T of tile i + 2 before O^T of tile i).
SV_DEVINL unsigned few_k(int i) { return i < 2 ? (unsigned)i : 2u * i - 2u; }
SV_DEVINL unsigned few_v(int i, int n) { return (unsigned)min(2 * i + 3, n + i); }

template <int RP, bool F8>
__global__ void __launch_bounds__(FewCfg<RP, F8>::kThreads, 1)
    tree_attn_few_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const __grid_constant__ TcArgs x) {
  using C = FewCfg<RP, F8>;
  constexpr int KT = 128, HR = C::HR, kSoft = C::kSoft;
  constexpr int kProducer = kSoft, kIssuer = kSoft + 1;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  unsigned char* pbuf = smem;                          // [tile of four][128 keys][128 bytes]
  unsigned char* ring = pbuf + 4 * C::kPBytes;
  unsigned char* qbuf = ring + C::kSlots * C::kSlot;   // [2 blocks][N1 rows][128 bytes]
  FewTail<RP>& f = *reinterpret_cast<FewTail<RP>*>(qbuf + C::kQBytes);
  TcTail& t = f.t;
  const Args& a = x.a;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int group = blockIdx.x;

  if (warp == 0) {
    find_range<KT>(x, t, group, lane);
  } else if (warp == kProducer && lane == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(smem_u32(&t.full[i]), 1);
      mbar_init(smem_u32(&t.empty[i]), 1);
    }
    mbar_init(smem_u32(&t.q_ready), kSoft);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&t.s_ready[i]), 1);
      mbar_init(smem_u32(&t.p_ready[i]), kSoft / 2);
      mbar_init(smem_u32(&t.pv_done[i]), 1);
    }
    mbar_init(smem_u32(&f.o_done), 1);
    mbar_init(smem_u32(&f.o_read), kSoft);
    t.abort = 0;
    t.bad[0] = t.bad[1] = t.badv[0] = t.badv[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&t.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_for_clear();
  fence_before();
  __syncthreads();
  fence_after();
  const unsigned tmem = t.tmem_base;
  volatile unsigned* abort = &t.abort;
  Walk<KT> w;
  w.start(a, t);

  if (warp == kProducer) {
    unsigned entry = 0;
    bool ok = true;
#pragma unroll 1
    for (; w.more() && ok; w.next(a)) {
      const int n = w.t1 - w.t0;
      int live = a.T;
      if (a.parents && (long long)w.t1 * KT > w.ctx) {
        live = 0;
        for (int i = lane; i < a.T; i += 32)
          if (a.parents[(long long)w.b * a.T + i] != -2) live = i + 1;
        live = __reduce_max_sync(0xffffffffu, live);
      }
      const bool seq_ok = ctx_ok(a, w.ctx);
      int nk = 0, nv = 0;  // keys and values issued
#pragma unroll 1
      for (int e = 0; e < 2 * n && ok; ++e, ++entry) {
        const bool isv = !(nk < n && nk < nv + 3);
        const int tile = w.t0 + (isv ? nv++ : nk++);
        const int pos = tile * KT + lane * x.box;
        int page = -1;
        if (seq_ok && lane < KT / x.box && pos < w.ctx + live && (pos >> x.lp) < a.max_pages)
          page = a.page_table[(long long)w.b * a.max_pages + (pos >> x.lp)];
        if (page < 0 || page >= a.num_pages) page = -1;
        const unsigned hit = __ballot_sync(0xffffffffu, page >= 0);
        const int s = (int)(entry % C::kSlots);
        ok = entry < (unsigned)C::kSlots ||
             warp_wait(smem_u32(&t.empty[s]), ((entry / C::kSlots) & 1) ^ 1, abort, a.status);
        if (!ok) break;
        const unsigned bar = smem_u32(&t.full[s]);
        const unsigned dst = smem_u32(ring + s * C::kSlot) + lane * x.box * 128;
        if (lane == 0) mbar_arrive_expect_tx(bar, (unsigned)__popc(hit) * x.box * (C::kSlot / KT));
        __syncwarp();
        if (page >= 0) {
          const CUtensorMap* map = isv ? &map_v : &map_k;
          tma_4d(dst, map, 0, 0, w.hk, page, bar);
          if (!F8) tma_4d(dst + KT * 128, map, 64, 0, w.hk, page, bar);
        }
      }
    }
    if (*abort) {  // copies in flight must land before the shared memory goes
      for (int i = 0; i < C::kSlots && entry >= (unsigned)i + 1; ++i) {
        const unsigned e = entry - 1 - i;
        const uint64_t t0 = global_ns();
        while (!mbar_test_parity(smem_u32(&t.full[e % C::kSlots]), (e / C::kSlots) & 1) &&
               global_ns() - t0 < 1000000) {
        }
      }
    }
  } else if (warp == kIssuer) {
    const unsigned lead = elect_lane();
    // fp32 accumulator, M = 128; A and B bf16 or e4m3 (code 0).
    constexpr uint32_t kTypes = F8 ? 0u : (1u << 7) | (1u << 10);
    constexpr uint32_t id_qk = (1u << 4) | kTypes | ((uint32_t)(C::N1 >> 3) << 17) | (8u << 24);
    constexpr uint32_t id_pv = (1u << 4) | kTypes | (1u << 15) | (1u << 16) | ((uint32_t)(C::N2 >> 3) << 17) | (8u << 24);
    const int ksteps = F8 ? (a.D + 31) / 32 : a.D / 16;
    const uint64_t q = desc_k(uni(smem_u32(qbuf)));
    unsigned entry0 = 0, item = 0, pcount[2] = {0, 0};
    bool ok = true;
    auto full = [&](unsigned e) {
      ok = ok && warp_wait(smem_u32(&t.full[e % C::kSlots]), (e / C::kSlots) & 1, abort, a.status);
      if (ok) fence_after();
      return ok;
    };
    auto qk = [&](int i) {
      const unsigned e = entry0 + few_k(i);
      if (!full(e)) return;
      const uint64_t k = desc_k(uni(smem_u32(ring + (e % C::kSlots) * C::kSlot)));
      const unsigned d = uni(tmem + C::kS + 128 * (i & 1));
      if (F8) {  // the pieces of Q one after the other
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((j & 3) < ksteps)
            mma_f8(lead, d, k + (j & 3) * 2, q + (j >> 2) * (C::N1 * 8) + (j & 3) * 2, id_qk, j > 0);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < ksteps)
            mma_ss(lead, d, k + (j >> 2) * (KT * 8) + (j & 3) * 2, q + (j >> 2) * (C::N1 * 8) + (j & 3) * 2, id_qk,
                   j > 0);
      }
      commit(lead, smem_u32(&t.s_ready[i & 1]));
      commit(lead, smem_u32(&t.empty[e % C::kSlots]));
    };
#pragma unroll 1
    for (; w.more() && ok; w.next(a), ++item) {
      const int n = w.t1 - w.t0;
      ok = ok && warp_wait(smem_u32(&t.q_ready), item & 1, abort, a.status);
      if (!ok) break;
      fence_after();
      qk(0);
      if (n > 1 && ok) qk(1);
#pragma unroll 1
      for (int i = 0; i < n && ok; ++i) {
        const int s = i & 1;
        ok = ok && warp_wait(smem_u32(&t.p_ready[s]), pcount[s] & 1, abort, a.status);
        // The warps of both streams read both streams' O of the last item; the first P comes
        // from the warps of one.
        if (i == 0 && item > 0) ok = ok && warp_wait(smem_u32(&f.o_read), (item - 1) & 1, abort, a.status);
        if (!ok) break;
        fence_after();
        ++pcount[s];
        if (i + 2 < n) qk(i + 2);
        const unsigned e = entry0 + few_v(i, n);
        if (!ok || !full(e)) break;
        const uint64_t v = desc_n(uni(smem_u32(ring + (e % C::kSlots) * C::kSlot)), KT * 128);
        const uint64_t p = desc_n(uni(smem_u32(pbuf + (i & 3) * C::kPBytes)), KT * 128);
        const unsigned d = uni(tmem + C::kO + 128 * s);
#pragma unroll
        for (int j = 0; j < (F8 ? 4 : 8); ++j) {
          const unsigned off = j * (F8 ? 4096 : 2048) >> 4;
          if (F8)
            mma_f8(lead, d, v + off, p + off, id_pv, i > 1 || j > 0);
          else
            mma_ss(lead, d, v + off, p + off, id_pv, i > 1 || j > 0);
        }
        commit(lead, smem_u32(&t.pv_done[s]));
        commit(lead, smem_u32(&t.empty[e % C::kSlots]));
      }
      if (ok) commit(lead, smem_u32(&f.o_done));
      entry0 += 2u * n;
    }
  } else if (warp < kSoft) {
    const int s = warp >> 3, h = warp >> 2 & 1, q = warp & 3;  // stream, half of the rows, 32 keys
    const int wt = threadIdx.x & 127;                          // key of the tile, and channel of the head
    const int st = threadIdx.x & 255;                          // thread of the stream
    const int row0 = h * HR;
    const unsigned lanes = (unsigned)(q * 32) << 16;
    const unsigned sbase = tmem + lanes + C::kS + 128 * s + h * C::HS;
    const unsigned obase = tmem + lanes + C::kO + 128 * s + h * C::HN;
    const int G = a.Hq / a.Hkv, nrows = x.rows;
    unsigned item = 0, scount = 0, entry0 = 0;
    auto wait = [&](unsigned long long* bar, unsigned parity) { bar_wait(smem_u32(bar), parity, abort, a.status); };

    // Q of an item: eight lanes a row, 16 values each; fetched early, stored when the
    // products with the last Q are done.
    const int qpos = threadIdx.x >> 3, qu = threadIdx.x & 7;  // row of the operand, 16 of its values
    const int qrow = qpos % C::HS < HR && qpos < C::N1 ? qpos / C::HS * HR + qpos % C::HS : RP;
    const bool q_on = qrow < nrows && qu * 16 < a.D;
    const long long q_at = q_on ? (long long)(qrow / G) * a.q_st + (long long)(qrow % G) * a.q_sh + qu * 16 : 0;
    uint4 qv[2];
    auto q_of = [&](const Walk<KT>& it) {
      return reinterpret_cast<const uint4*>(a.q + it.b * a.q_sb + (long long)it.hk * G * a.q_sh + q_at);
    };
    auto fetch_q = [&](const Walk<KT>& it) {
      qv[0] = qv[1] = make_uint4(0, 0, 0, 0);
      if (q_on && !x.qzero) {
        qv[0] = q_of(it)[0];
        qv[1] = q_of(it)[1];
      }
    };
    auto put_q = [&](unsigned parity) {
      uint32_t z[8] = {qv[0].x, qv[0].y, qv[0].z, qv[0].w, qv[1].x, qv[1].y, qv[1].z, qv[1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] ^= x.qflip;
      float down = 1.0f;
      if (F8) {
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(z[j])), fabsf(bf16_hi(z[j]))));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^e with top 2^e in (224, 448]; rows of zeros or with infinities as they are.
        const unsigned bits = __float_as_uint(top);
        int e = ((bits & 0x7fffffu) > 0x600000u ? 134 : 135) - (int)(bits >> 23);
        if (!(top > 0.0f) || !(top < INFINITY)) e = 0;
        e = max(-126, min(126, e));
        const float up = __int_as_float((e + 127) << 23);
        down = __int_as_float((127 - e) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y0 = bf16_lo(z[j]) * up, y1 = bf16_hi(z[j]) * up;
          const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
          const float2 back = __half22float2(e4m3_to_half2(c));
          const uint32_t l =
              __nv_cvt_float2_to_fp8x2(make_float2(y0 - back.x, y1 - back.y), __NV_SATFINITE, __NV_E4M3);
          // e4m3 has no infinity: an infinite element counts as NaN.
          const uint32_t nan = (isfinite(y0) ? 0u : 0x7fu) | (isfinite(y1) ? 0u : 0x7f00u);
          if (j & 1) {
            hi[j >> 1] |= (c | nan) << 16;
            lo[j >> 1] |= (l | nan) << 16;
          } else {
            hi[j >> 1] = c | nan;
            lo[j >> 1] = l | nan;
          }
        }
        if (qpos < C::N1) {
          unsigned char* at = qbuf + qpos * 128 + ((qu ^ (qpos & 7)) << 4);
          *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(at + C::N1 * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      } else if (qpos < C::N1) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int c = 2 * qu + k;
          *reinterpret_cast<uint4*>(qbuf + (c >> 3) * C::N1 * 128 + qpos * 128 + (((c & 7) ^ (qpos & 7)) << 4)) =
              make_uint4(z[4 * k], z[4 * k + 1], z[4 * k + 2], z[4 * k + 3]);
        }
      }
      if (qu == 0 && qrow < RP) f.qc[parity][qrow] = x.c * down;
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&t.q_ready));
    };
    // Page of this thread's key in tile i of an item, -1 for none, and the key's scales.
    auto page_of = [&](const Walk<KT>& it, int i) -> int {
      const long long pos = (long long)(it.t0 + i) * KT + wt;
      if (!ctx_ok(a, it.ctx) || it.t0 + i >= it.t1 || pos >= (long long)it.ctx + a.T ||
          (pos >> x.lp) >= a.max_pages)
        return -1;
      return a.page_table[(long long)it.b * a.max_pages + (pos >> x.lp)];
    };
    auto scales_of = [&](const Walk<KT>& it, int i, int id, float* k, float* v) {
      *k = *v = 0.0f;
      if (!F8 || id < 0 || id >= a.num_pages) return;
      const long long at =
          (((long long)id * a.Hkv + it.hk) << x.lp) + (((it.t0 + i) * KT + wt) & (a.P - 1));
      *k = __ldg(a.ks + at);
      *v = __ldg(a.vs + at);
    };
    // A tile's scales are fetched two of the stream's tiles ahead, its page three.
    int id = -1, id1 = -1, id2 = -1;
    float ksc = 0.0f, vsc = 0.0f, ksc1 = 0.0f, vsc1 = 0.0f;
    if (threadIdx.x < RP) f.row_out[threadIdx.x] = threadIdx.x / G * a.Hq + threadIdx.x % G;
    if (w.more()) {
      id = page_of(w, s);
      id1 = page_of(w, s + 2);
      id2 = page_of(w, s + 4);
      fetch_q(w);
      scales_of(w, s, id, &ksc, &vsc);
      scales_of(w, s + 2, id1, &ksc1, &vsc1);
      put_q(0);
    }

#pragma unroll 1
    for (; w.more(); ++item) {
      const int n = w.t1 - w.t0;
      const bool seq_ok = ctx_ok(a, w.ctx);
      const bool tail = seq_ok && (long long)w.t1 * KT > w.ctx;
      int* par = t.par[item & 1][s];
      unsigned long long* anc = f.anc[item & 1][s];
      const float* qc = f.qc[item & 1] + row0;
      const float* mref = f.mref[s] + row0;
      if (st < RP) f.mref[s][st] = st < nrows ? kNoScore : -kNoScore;  // (no score of 0 exceeds that)
      unsigned bad = seq_ok ? 0u : (unsigned)SV_DEV_PAGE_RANGE;
      if (tail && st < a.T) par[st] = a.parents ? a.parents[(long long)w.b * a.T + st] : st - 1;
      // The next item's first needs on their way to L2 while this one is worked on.
      {
        Walk<KT> nx = w;
        nx.next(a);
        if (nx.more() && q_on) asm volatile("prefetch.global.L2 [%0];" ::"l"(q_of(nx)));
      }
      named_sync(1 + s, 256);
      if (tail) {
        if (st < a.T) {
          const int p = par[st];
          if (p < -2 || p >= st || (p >= 0 && par[p] == -2)) bad |= SV_DEV_TREE;
          unsigned long long set = 0;
#pragma unroll 1
          for (int j = st, left = a.T; j >= 0 && left > 0; --left) {
            const int pj = par[j];
            if (pj == -2) break;
            set |= 1ull << j;
            j = pj < j ? pj : -1;
          }
          anc[st] = set;
        }
        named_sync(1 + s, 256);
      }

      float l[HR];
#pragma unroll
      for (int r = 0; r < HR; ++r) l[r] = 0.0f;
      bool any = false;
#pragma unroll 1
      for (int i = s; i < n; i += 2) {
        const int tile = w.t0 + i;
        const bool edge = (long long)(tile + 1) * KT > w.ctx || !seq_ok;
        // Rows of the half that attend this thread's key.
        unsigned see = ~0u;
        const long long nd = (long long)tile * KT + wt - w.ctx;  // the key's node
        if (edge) {
          unsigned long long all = ~0ull;
          if (!seq_ok || nd >= a.T) {
            all = 0;
          } else if (nd >= 0) {
            all = 0;
#pragma unroll 1
            for (int k = (int)nd; k < a.T; ++k)  // a node's descendants come after it
              if (anc[k] >> nd & 1ull) all |= ((1ull << G) - 1) << (k * G);
          }
          see = (unsigned)(all >> row0);
        }
        // A needed page outside the cache or the table; then the next pages and scales.
        if (seq_ok && (nd < 0 || (nd < a.T && par[nd] != -2)) && (id < 0 || id >= a.num_pages))
          bad |= SV_DEV_PAGE_RANGE;
        const float kc = F8 ? ksc : 1.0f;
        const float vs = F8 ? vsc * C::kLift : 1.0f;
        const float lv = F8 ? __log2f(fmaxf(vsc, kLeastScale)) : 0.0f;
        id = id1;
        if (F8) {
          ksc = ksc1;
          vsc = vsc1;
          scales_of(w, i + 4, id2, &ksc1, &vsc1);
          id1 = id2;
          id2 = page_of(w, i + 6);
        } else {
          id1 = page_of(w, i + 4);
        }

        wait(&t.s_ready[s], scount & 1);
        fence_after();
        // Scores less m, in powers of two; masked ones -inf.
        float y[C::HS];
        auto scores = [&](bool less) {
          tmem_ld_cols<C::HS>(sbase, y);
#pragma unroll
          for (int r = 0; r < HR; r += 4) {
            const float4 c4 = *reinterpret_cast<const float4*>(qc + r);
            const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
            float mm[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (less) {
              const float4 m4 = *reinterpret_cast<const float4*>(mref + r);
              mm[0] = m4.x;
              mm[1] = m4.y;
              mm[2] = m4.z;
              mm[3] = m4.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) y[r + j] = __fmaf_rn(y[r + j], F8 ? cc[j] * kc : cc[j], -mm[j]);
          }
          if (edge) {
#pragma unroll
            for (int r = 0; r < HR; ++r) y[r] = see >> r & 1u ? y[r] : -INFINITY;
          }
        };
        scores(true);
        float over[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int r = 0; r < HR; ++r) over[r & 3] = fmaxf(over[r & 3], y[r]);
        const bool up = fmaxf(fmaxf(over[0], over[1]), fmaxf(over[2], over[3])) > C::kGrow - lv;
        const bool raise = named_any(1 + s, 256, up);
        // (This tile's P buffer is free: its S^T was issued, and announced, after the
        // product that read the buffer four tiles ago.)
        if (raise) {
          if (any) {  // O of this stream: its last product must be complete
            wait(&t.pv_done[s], (scount - 1) & 1);
            fence_after();
          }
          // New references: the stream's maxima; then O and the sums to match.
          scores(false);
          {
            float v[HR];
#pragma unroll
            for (int r = 0; r < HR; ++r) v[r] = y[r] + lv;
            halve<true, HR, 16>(v, lane, 0, HR, f.wmax[s][q] + row0);
          }
          named_sync(1 + s, 256);
          if (st < RP) {
            const float top = fmaxf(fmaxf(f.wmax[s][0][st], f.wmax[s][1][st]),
                                    fmaxf(f.wmax[s][2][st], f.wmax[s][3][st]));
            const float old = f.mref[s][st];
            float fr = 1.0f;
            if (st < nrows && top > old) {  // every row that grew, so that the next raise is far
              f.mref[s][st] = top;
              fr = ex2_fast(old - top);
            }
            f.fac[s][st] = fr;
          }
          named_sync(1 + s, 256);
          const float* fac = f.fac[s] + row0;
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            l[r] *= fac[r];
            y[r] -= mref[r];
          }
          if (any) {
#pragma unroll 1
            for (int r = 0; r < HR; r += 4) {
              const float4 f4 = *reinterpret_cast<const float4*>(fac + r);
#pragma unroll
              for (int pc = 0; pc < (F8 ? 3 : 1); ++pc) {
                float v[4];
                tmem_ld4(obase + pc * HR + r, v);
                tmem_st4(obase + pc * HR + r, v[0] * f4.x, v[1] * f4.y, v[2] * f4.z, v[3] * f4.w);
              }
            }
            tmem_wait_st();
          }
          named_sync(1 + s, 256);  // fac has been read
        }
        // Weights, their sums, and P^T: the half's part of this key's 128 bytes.
        constexpr int kWords = C::HN / (F8 ? 4 : 2);
        uint32_t words[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) words[k] = 0;
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          float p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = ex2_fast(y[r + j]);
            l[r + j] += p[j];
          }
          if (F8) {
            const float2 p0 = f2_mul(make_float2(p[0], p[1]), f2(vs)), p1 = f2_mul(make_float2(p[2], p[3]), f2(vs));
            p[0] = p0.x;
            p[1] = p0.y;
            p[2] = p1.x;
            p[3] = p1.y;
            if (edge) {  // the scale may be NaN
#pragma unroll
              for (int j = 0; j < 4; ++j) p[j] = see >> (r + j) & 1u ? p[j] : 0.0f;
            }
            const __half2 step = __half2half2(__ushort_as_half(0x5000));  // 32
            uint32_t c[3][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const __half2 w0 = __floats2half2_rn(p[2 * j], p[2 * j + 1]);
              c[0][j] = half2_to_e4m3(w0);
              const __half2 r1 = __hmul2(__hsub2(w0, e4m3_to_half2(c[0][j])), step);
              c[1][j] = half2_to_e4m3(r1);
              const __half2 r2 = __hmul2(__hsub2(r1, e4m3_to_half2(c[1][j])), step);
              c[2][j] = half2_to_e4m3(r2);
            }
            words[r / 4] = __byte_perm(c[0][0], c[0][1], 0x5410);
            words[(HR + r) / 4] = __byte_perm(c[1][0], c[1][1], 0x5410);
            words[(2 * HR + r) / 4] = __byte_perm(c[2][0], c[2][1], 0x5410);
          } else {
            words[r / 2] = pack_bf16(p[0], p[1]);
            words[r / 2 + 1] = pack_bf16(p[2], p[3]);
          }
        }
        unsigned char* prow = pbuf + (i & 3) * C::kPBytes + wt * 128;
        const int unit0 = h * (kWords / 4);
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k)
          *reinterpret_cast<uint4*>(prow + (((unit0 + k) ^ (wt & 7)) << 4)) =
              make_uint4(words[4 * k], words[4 * k + 1], words[4 * k + 2], words[4 * k + 3]);
        if (edge) {
          // 0 times what lies at masked positions must be 0: rows past the tree are zeroed, a
          // node's NaN (or infinity) is taken out and given to its descendants at the end.
          const unsigned ev = entry0 + few_v(i, n);
          wait(&t.full[ev % C::kSlots], (ev / C::kSlots) & 1);
          if (nd >= 0 || !seq_ok) {
            unsigned char* vrow = ring + (ev % C::kSlots) * C::kSlot + wt * 128;
            const bool dead = !seq_ok || nd >= a.T || par[nd] == -2;
#pragma unroll 2
            for (int u = h * (F8 ? 4 : 8); u < (h + 1) * (F8 ? 4 : 8); ++u) {
              uint4* at = reinterpret_cast<uint4*>(vrow + (u >> 3) * KT * 128 + (((u & 7) ^ (wt & 7)) << 4));
              uint4 v = dead ? make_uint4(0, 0, 0, 0) : *at;
              uint32_t z[4] = {v.x, v.y, v.z, v.w}, found = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                // Top bits of the bytes or halves whose element is not finite: those whose
                // exponent (and mantissa, of a code) are all ones, difference zero.
                const uint32_t ones = F8 ? 0x7f7f7f7fu : 0x7f807f80u;
                const uint32_t top = F8 ? 0x80808080u : 0x80008000u;
                const uint32_t m = ~(((z[j] & ones) ^ ones) + (top - (F8 ? 0x01010101u : 0x00010001u))) & top;
                z[j] &= ~(F8 ? (m >> 7) * 0xffu : (m >> 15) * 0xffffu);
                found |= m;
              }
              if (found) t.badv[item & 1] = 1;
              if (found || dead) *at = make_uint4(z[0], z[1], z[2], z[3]);
            }
          }
        }
        fence_async();
        any = true;
        ++scount;
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(smem_u32(&t.p_ready[s]));
      }
      entry0 += 2u * n;

      // ---- the item's end
      Walk<KT> nx = w;
      nx.next(a);
      if (nx.more()) {
        fetch_q(nx);
        id = page_of(nx, s);
        id1 = page_of(nx, s + 2);
        id2 = page_of(nx, s + 4);
      }
      if (bad) {
        atomicOr(&t.bad[item & 1], 1u);
        atomicOr(a.status, bad);
      }
      halve<false, HR, 16>(l, lane, 0, HR, f.wsum[s][q] + row0);
      named_sync(3, 32 * kSoft);
      // The next item's flags are cleared between the two barriers: the last item's, in the
      // same place, were read before its second one, and the next sets them after this one's.
      if (threadIdx.x == 0) t.bad[(item + 1) & 1] = t.badv[(item + 1) & 1] = 0;
      // Both streams have read their last S: the next item's Q may go in.
      if (nx.more()) {
        put_q((item + 1) & 1);
        scales_of(nx, s, id, &ksc, &vsc);
        scales_of(nx, s + 2, id1, &ksc1, &vsc1);
      }
      const bool at_fault = t.bad[item & 1] != 0, badv = t.badv[item & 1] != 0;
      if (threadIdx.x < RP) {
        const int r = threadIdx.x;
        const bool dead = r < nrows && a.parents && a.parents[(long long)w.b * a.T + r / G] == -2;
        const float m0 = f.mref[0][r], m1 = n > 1 ? f.mref[1][r] : kNoScore;
        const float m = fmaxf(m0, m1);
        const float g0 = ex2_fast(m0 - m), g1 = n > 1 ? ex2_fast(m1 - m) : 0.0f;
        const float l0 = (f.wsum[0][0][r] + f.wsum[0][1][r]) + (f.wsum[0][2][r] + f.wsum[0][3][r]);
        const float l1 = (f.wsum[1][0][r] + f.wsum[1][1][r]) + (f.wsum[1][2][r] + f.wsum[1][3][r]);
        const float sum = dead ? 0.0f : l0 * g0 + (n > 1 ? l1 * g1 : 0.0f);
        const bool whole = w.t0 == 0 && w.t1 == w.n;
        // Factors of the streams' O: for a whole item with the division by the sum.
        float inv = 1.0f;
        if (whole) inv = at_fault ? __int_as_float(0x7fc00000) : sum == 0.0f ? 0.0f : 1.0f / sum;
        f.fin[r] = make_float4(g0 / C::kLift, g1 / C::kLift,
                               whole ? inv : at_fault ? __int_as_float(0x7fc00000) : m, sum);
      }
      // (pv_done's parity would not do here: a tile's S^T is issued before the product of the
      // stream's tile before it, so that two of them may be outstanding.)
      wait(&f.o_done, item & 1);
      fence_before();
      named_sync(3, 32 * kSoft);
      fence_after();
      const bool whole = w.t0 == 0 && w.t1 == w.n;
      const long long slot = (long long)group * 2 + (w.t0 == 0 ? 1 : 0);
      // A row a group of four warps and step (a short loop: it runs once an item).
      const long long out0 = ((long long)w.b * a.T * a.Hq + w.hk * G) * a.D + wt;
#pragma unroll 2
      for (int r = 2 * s + h; r < nrows; r += 4) {
        __syncwarp();  // tensor memory is read by whole warps
        const float4 fin = f.fin[r];
        const unsigned col = tmem + lanes + C::kO + (r >= HR ? C::HN + r - HR : r);
        float o0, o1 = 0.0f;
        if (F8) {
          float u[6];
          tmem_ld_3x2(col, HR, 128, u);
          o0 = __fmaf_rn(__fmaf_rn(u[2], 0.03125f, u[1]), 0.03125f, u[0]);
          o1 = __fmaf_rn(__fmaf_rn(u[5], 0.03125f, u[4]), 0.03125f, u[3]);
        } else {
          tmem_ld_1x2(col, 128, &o0, &o1);
        }
        float v = o0 * fin.x;
        if (n > 1) v = __fmaf_rn(o1, fin.y, v);  // (else the second stream had no tile)
        if (wt >= a.D) continue;
        if (badv) {  // NaN and infinities of the nodes the row attends
          for (int k = 0; k < a.T; ++k) {
            const long long pos = (long long)w.ctx + k;
            if (pos < (long long)w.t0 * KT || pos >= (long long)w.t1 * KT || (pos >> x.lp) >= a.max_pages) continue;
            const int pg = a.page_table[(long long)w.b * a.max_pages + (pos >> x.lp)];
            if (pg < 0 || pg >= a.num_pages || !(anc[r / G] >> k & 1ull)) continue;
            const long long at = (((long long)pg * a.Hkv + w.hk) * a.P + (pos & (a.P - 1))) * a.D + wt;
            const float z = F8 ? ((static_cast<const unsigned char*>(a.vc)[at] & 0x7f) == 0x7f
                                      ? __int_as_float(0x7fc00000)
                                      : 0.0f)
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.vc)[at]);
            if (!isfinite(z)) v += z;
          }
        }
        if (whole) {
          a.out[out0 + (long long)f.row_out[r] * a.D] = __float2bfloat16_rn(fin.z == 0.0f ? 0.0f : v * fin.z);
        } else {
          x.part_o[(slot * nrows + r) * a.D + wt] = v;
          if (wt == 0) x.part_ml[slot * nrows + r] = make_float2(fin.z, fin.w);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&f.o_read));
      if (!whole)
        join_parts(x, t, w, 0, nrows, nrows, 32 * kSoft);
      w = nx;
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kIssuer) {
    __syncwarp();
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// Clears the status word and the counters of parts. The attention kernel starts while it
// runs (what came before it in the stream has ended by then), and waits for its end
// before any of them is touched.
__global__ void clear_kernel(unsigned* p, int n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0;
}

// ---------------------------------------------------------------- any shape
//
// One warp a query row, one key at a time, running maximum and sum in fp32.
// Takes every head size and page size; bound by the latency of a key's
// reduction over the lanes: 8 sequences of 4 nodes, 32 heads of 100, 2000 keys, e4m3: 2.7 ms.

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
    const int need = (int)(((long long)ctx + live + a.P - 1) / a.P);
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
  return (long long)max_pages * page_size < (1ll << 31) - 2 * kTreeMax &&
         (long long)B * T * Hq < (1ll << 31) && (long long)B * max_pages < (1ll << 40);
}

// Shapes that the tensor-core kernel takes.
bool tc_shape(int D, int page_size) {
  return D % 16 == 0 && D <= 256 && (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128);
}

// How the rows of an item are cut: up to 128 in one Q tile; more in pairs of equal
// tiles (D above 128: single tiles), a CTA each.
struct Plan {
  int rows, rpt, parts, groups, cta_rows;
  bool shared;
  size_t off_counters, off_ml, off_o, total;
};

Plan make_plan(int T, int Hq, int Hkv, int D) {
  Plan p{};
  p.rows = T * (Hq / Hkv);
  p.shared = D <= 128 && p.rows > 128;
  if (p.shared) {
    p.parts = (p.rows + 255) / 256;
    p.rpt = (p.rows + 2 * p.parts - 1) / (2 * p.parts);
    p.cta_rows = 2 * p.rpt;
  } else {
    p.parts = (p.rows + 127) / 128;
    p.rpt = (p.rows + p.parts - 1) / p.parts;
    p.cta_rows = p.rpt;
  }
  p.groups = std::max(1, kMaxCtas / p.parts);
  const size_t slots = (size_t)p.groups * p.parts * 2;
  size_t off = 256;
  p.off_counters = off;
  off = align_up(off + (size_t)p.groups * p.parts * 4, 256);
  p.off_ml = off;
  off = align_up(off + slots * p.cta_rows * sizeof(float2), 256);
  p.off_o = off;
  off = align_up(off + slots * p.cta_rows * (size_t)D * 4, 256);
  p.total = off;
  return p;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The cache as boxes of `box` tokens of one page and head: bf16 in columns of 64
// with the 128-byte swizzle, codes in whole rows of DP.
bool make_map(CUtensorMap* m, const void* base, const Args& a, bool f8, int dp, int box, bool swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  const size_t es = f8 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.P, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  const cuuint64_t strides[3] = {a.D * es, (cuuint64_t)a.P * a.D * es, (cuuint64_t)a.Hkv * a.P * a.D * es};
  const cuuint32_t boxes[4] = {(cuuint32_t)(f8 ? dp : 64), (cuuint32_t)box, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A launch that may begin before the kernel ahead of it has ended.
template <typename Kernel>
int launch_early(Kernel kernel, unsigned grid, int threads, int smem, cudaStream_t st, const CUtensorMap& mk,
                 const CUtensorMap& mv, const TcArgs& x) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mk, mv, x) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

template <int DP, bool F8, bool SHARED>
int launch_tc(const TcArgs& x, cudaStream_t st) {
  constexpr int kSmem = tc_smem<DP, F8, SHARED>();
  static std::mutex mu;
  static bool set[64] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[device]) {
      if (cudaFuncSetAttribute(tree_attn_kernel<DP, F8, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmem) != cudaSuccess)
        return SV_ERR_CUDA;
      set[device] = true;
    }
  }
  CUtensorMap mk, mv;
  if (!make_map(&mk, x.a.kc, x.a, F8, DP, x.box, !F8) || !make_map(&mv, x.a.vc, x.a, F8, DP, x.box, !F8))
    return SV_ERR_CUDA;
  return launch_early(tree_attn_kernel<DP, F8, SHARED>, (unsigned)(x.groups * x.parts_per_item),
                      Cfg<DP, F8, SHARED>::kThreads, kSmem, st, mk, mv, x);
}

template <int RP, bool F8>
int launch_few(const TcArgs& x, cudaStream_t st) {
  constexpr int kSmem = few_smem<RP, F8>();
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static std::mutex mu;
  static bool set[64] = {};
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || device < 0 || device >= 64) return SV_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[device]) {
      if (cudaFuncSetAttribute(tree_attn_few_kernel<RP, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmem) != cudaSuccess)
        return SV_ERR_CUDA;
      set[device] = true;
    }
  }
  CUtensorMap mk, mv;
  if (!make_map(&mk, x.a.kc, x.a, F8, 128, x.box, true) || !make_map(&mv, x.a.vc, x.a, F8, 128, x.box, true))
    return SV_ERR_CUDA;
  return launch_early(tree_attn_few_kernel<RP, F8>, (unsigned)x.groups, FewCfg<RP, F8>::kThreads, kSmem, st, mk, mv,
                      x);
}

// Whether keys, not rows, are the M of the products. Measured, keys / rows as M in us:
// e4m3, 64 sequences to 8192, D 128: 159 / 403 (4 rows), 205 / 409 (36), since only the
// first takes the codes as they are; it loses only for contexts of a few tiles (53 / 48
// at 300 keys, 36 rows, D 64). bf16, D 128: one sequence of 32768 37 / 42 (4 rows) and 52 / 54
// (36); 64 to 8192 205 / 202 and 222 / 209; 160 to 1024 111 / 122 and 148 / 139. bf16, D 64,
// one sequence of 32768 31 / 28 and 41 / 35; 64 to 8192 175 / 131 and 200 / 136.
bool keys_as_m(int rows, int D, bool f8) {
  return f8 ? D <= 128 && rows <= kFewRows : D > 64 && D <= 128 && rows <= 16;
}

template <bool F8>
int launch_tc_any(TcArgs& x, const Plan& p, cudaStream_t st) {
  const int D = x.a.D;
  x.box = std::min(x.a.P, D > 128 ? 64 : 128);
  x.lp = x.a.P == 16 ? 4 : x.a.P == 32 ? 5 : x.a.P == 64 ? 6 : 7;
  if (keys_as_m(p.rows, D, F8)) {
    if constexpr (F8) {
      if (p.rows > 16) return launch_few<kFewRows, true>(x, st);
    }
    return launch_few<16, F8>(x, st);
  }
  if (D > 128) return launch_tc<256, F8, false>(x, st);
  if (D > 64) return p.shared ? launch_tc<128, F8, true>(x, st) : launch_tc<128, F8, false>(x, st);
  return p.shared ? launch_tc<64, F8, true>(x, st) : launch_tc<64, F8, false>(x, st);
}

}  // namespace tat
}  // namespace sv

using namespace sv::tat;

extern "C" {

size_t sv_tree_attention_workspace_size(int B, int T, int Hq, int Hkv, int D, int max_pages,
                                        int page_size) {
  if (!sizes_ok(B, T, Hq, Hkv, D, max_pages, page_size)) return 0;
  return tc_shape(D, page_size) ? make_plan(T, Hq, Hkv, D).total : 256;
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
  // 16-byte aligned rows for the tensor-core kernel; scales are copied in 16 bytes too.
  const bool tc = tc_shape(D, page_size) && !misaligned(q, 16) && !misaligned(out, 16) &&
                  !misaligned(k_cache, 16) && !misaligned(v_cache, 16) && !misaligned(k_scale, 16) &&
                  !misaligned(v_scale, 16) && q_stride_b % 8 == 0 && q_stride_t % 8 == 0 && q_stride_h % 8 == 0;
  if (tc) {
    const Plan p = make_plan(T, Hq, Hkv, D);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    TcArgs x{};
    x.a = a;
    x.rows = p.rows;
    x.rpt = p.rpt;
    x.parts_per_item = p.parts;
    x.groups = p.groups;
    x.c = scale == 0.0f ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
    x.join_c = keys_as_m(p.rows, D, cache_dtype == SV_E4M3) ? 1.0f : x.c;
    x.qflip = scale < 0.0f ? 0x80008000u : 0u;
    x.qzero = scale == 0.0f;
    x.counters = reinterpret_cast<unsigned*>(ws + p.off_counters);
    x.part_ml = reinterpret_cast<float2*>(ws + p.off_ml);
    x.part_o = reinterpret_cast<float*>(ws + p.off_o);
    clear_kernel<<<1, 256, 0, st>>>(static_cast<unsigned*>(workspace), (int)(p.off_ml / 4));
    if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
    return cache_dtype == SV_E4M3 ? launch_tc_any<true>(x, p, st) : launch_tc_any<false>(x, p, st);
  }
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
