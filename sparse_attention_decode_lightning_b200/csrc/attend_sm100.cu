// MLA decode attention over a list of cached tokens, on sm_100a tensor cores:
// the window-and-sinks and the block-scaled selected forms.  Per head h of
// query q, over the tokens j of its list:
//   z_j = scale * q[h, 0:576] . C[j, 0:576],  O[h] = sum_j softmax(z)_j C[j, 0:512],
//   LSE[h] = ln sum_j exp(z_j);   an empty list gives O = 0, LSE = -inf.
// The list is the first `sinks` and the last `window` visible positions
// (RANGE), or a row of selected positions (IDX).  The cache is bf16, or e4m3
// codes with an fp32 scale s_j for each block of tokens: C[j] = s_j * code[j].
//
// One pass over the list in tiles of 128 tokens by a cluster of two CTAs and
// cta_group::2 MMAs (M = 128 over the pair).  A CTA owns half of the heads as
// accumulator rows, the scores' keys of 64 of the tile's tokens, and 256 of the
// 512 value dims of all 128, so nothing is computed twice and neither scores
// nor P cross between the CTAs:
//   scores  D[64 heads x 128 tokens] a CTA: 36 steps of N = 128
//   values  D[64 heads x 512 dims]   a CTA: 8 steps of 2 x N = 256
// About 2200 tensor cycles a tile.  A CTA alone would have to hold the query of
// all heads (144 KB), or read every token for each half of them.
//
// The work is cut evenly: the tiles of all queries, one after another, are
// divided over the SM pairs, so ragged lists leave no pair idle; where there are
// enough of them a query counts START tiles more, what beginning one costs.  A
// query whose tiles lie on several pairs leaves partial results that a second
// kernel merges by log-sum-exp.
//
// Operands.  bf16 cache: q, C and P as bf16 (P's rounding, 2^-9 of each
// weight, is the size of the output's own).  e4m3 cache: codes widened to fp16
// (exact), q scaled by a power of two a head so that its largest element lies
// in [2^14, 2^15) and rounded to fp16 (exact for all that is not 2^-28 times
// smaller), P as fp16.  The scales enter in fp32, token by token: with
//   z_j = log2(e) scale q . code_j s_j + log2 s_j,
//   P_j = 2^(z_j - m + 7) = weight_j s_j 2^7 / 2^m,   l = sum P_j / s_j,
// O = P code / l.  m follows the largest z, that is the largest product of a weight
// and its scale, and may lag by 8: that token's P lies in [2^7, 2^15], fp16's upper
// end.  Another's keeps 11 bits down to 2^-14, so as long as weight x scale is at
// least 2^-21 of the largest, and is lost below 2^-32 of it.  (One scale a tile, its
// largest, with factors s_j / s in P, saves an addition but lost every weight of a
// tile in which another token's scale is much larger.)  Sums, maxima and O are fp32.
//
// Tensor memory (512 columns): O [0,256), lanes 0..63 dims 0..255 of the CTA's
// heads, lanes 64..127 dims 256..511 | scores slot 0 [256,320) | slot 1
// [320,384).  Shared memory: the query (72 KB), P (16 KB), the rings of keys and
// values in the 128-byte swizzle, refilled as soon as their MMAs have read them:
//   bf16   keys three groups of 3 chunks (64 tokens x 64 dims), values three
//          units of 32 tokens x 256 dims, all filled by TMA
//   e4m3   raw units by TMA (keys 64 tokens x 256 and x 320 codes, values 2 x 32
//          tokens x 256 codes), widened into two slots of 2 chunks, one of the
//          positions, and two value units
// A load costs about 45 cycles to issue whatever it brings (a gather of four rows
// 57), so 16 rows that are consecutive in the pool come as one box (of the bf16
// keys 8), others by gathers of four.  Rows that the list does not hold are
// loaded from outside the pool, as zeros, and never read, so that what lies in
// the cache there (NaN, say) cannot reach a product.  For the same reason two
// queries of 64 heads do not share a tile: a token that one of them lists would
// meet the other's zero weight.  TMA carries all of it: the same loads issued by
// threads (cp.async, or registers) fill the load/store unit's queue, behind which
// every barrier and fence of the SM waits; a tile took 10,500 cycles that way.
//
// Roles, by warp:
//   0       score MMAs of both CTAs (in the first)      1  loads queries and keys
//   2       loads values      3  looks up pool rows (list -> page table -> scale),
//           the loads of three tiles under way at once, and sends the rows to L2
//   4..11   softmax, rescale and output, a row's 128 tokens and 512 dims in four
//           parts, one a thread, which exchange their maxima
//   bf16: 12 value MMAs; e4m3: 12..19 widen keys and scale the query, 20..23 widen
//   values, 24 value MMAs
// The two sorts of MMAs have a warp each, since waiting and issuing take longer
// than the MMAs themselves (one warp for both: 24 verifying users 47.4 against
// 45.1 us), and so that scores run up to two tiles ahead.  Widening the keys was the
// longest chain, so two groups of four warps take turns at it (32 users, windows of
// 4096: 72.6 -> 69.5 us).
//
// What bounds it.  bf16: a tile takes about 4200 cycles on a pair, its 147 KB from
// DRAM at a 74th of the copy rate 3100; the rings, all the shared memory there
// is, hold one tile, so a load's latency is not quite covered.  16 users, 128 heads,
// windows of 8192: 56.1 us, 2.4 TB/s.  e4m3: about 5300 cycles, of which the MMAs
// are 2200; shared memory moves some 4000 cycles' worth a tile (the widening reads 1 and
// writes 2 bytes a code, MMAs read 4 for it), the softmax is busy for 3600.  4 users,
// 128 heads, dense over 131072 tokens: 213 us, 685 TFLOP/s, 1.4 TB/s of codes.
// What a call takes beside its tiles, from a fit over 2 to 16 tiles on every pair (a
// query a pair, replayed as a graph): 11.2 us + 2.4 a tile over bf16, 14.7 + 3.1 over
// e4m3 (64 heads: 9.4 and 13.5), and 2 more where a query is divided: the shares, the
// first look-up (three dependent loads), cold instructions (the hot code is kept below
// 60 KB: past the instruction cache every warp slows down several times), output, merge.
// The launch itself, barriers and tensor memory come beside the end of the kernel before
// (programmatic serialization): one user's selected step 27.0 -> 24.6 us.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace dsa {
namespace {

constexpr int NT = 128;                              // tokens per tile
constexpr int NH = NT / 2;                           // of them keys of one CTA
constexpr int RH = 64;                               // accumulator rows (heads) a CTA
constexpr int CH = 64 * 128;                         // chunk bytes: 64 rows x 64 dims x 2
constexpr int KC = DSA_DIM / 64;                     // chunks of a row of 576
constexpr int VT = 32;                               // tokens of a value unit
constexpr int VCH = 16 * 128;                        // bytes of 16 tokens x 64 dims
constexpr int VSTEP = 4 * VCH;                       // and x 256 dims: one MMA step
constexpr int VSLOT = VT / 16 * VSTEP;
constexpr int VS = NT / VT;                          // units a tile takes
constexpr int KU = 2;                                // units of a tile's key codes: 256 dims, 320 dims
constexpr int KUB = NH * 256;                        // bytes of the first
constexpr int VUB = VT * 256;                        // bytes of a value unit's codes
constexpr int VUR = 2;                               // units of their ring
constexpr int RUN = 16;                              // rows that one load can bring where they are consecutive
constexpr int START = 2;                              // tiles that beginning a query costs
constexpr int RR = 4;                                // tiles looked up ahead
constexpr int QM = 4;                                // queries whose factors are kept
constexpr int SMX = 8;                               // softmax warps
constexpr int GROUP = 4;                             // warps that widen keys; as many widen values
constexpr int SMX0 = 4;                              // first of the softmax warps

template <bool KV8>
struct Plan {
  static constexpr int WARPS = SMX0 + SMX + (KV8 ? 4 * GROUP : 1);
  static constexpr int THREADS = 32 * WARPS;
  // A tile's 9 key chunks come in groups, each with its slot: three of three, or
  // (e4m3) four of two, through two slots, and the positions.
  static constexpr int KG = KV8 ? 5 : 3;
  static constexpr int KS = 3;                       // slots
  static constexpr int KCH = KV8 ? 2 : 3;            // chunks of a slot
  static constexpr int VR = KV8 ? 2 : 3;             // units of the value ring
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + KC * CH;
  static constexpr int OFF_V = OFF_K + (KV8 ? 5 : 9) * CH;
  static constexpr int OFF_P = OFF_V + VR * VSLOT;   // [2][64 heads x 64 tokens]
  static constexpr int OFF_KU = OFF_P + 2 * CH;      // e4m3: units of a tile's keys
  static constexpr int OFF_VU = OFF_KU + (KV8 ? NH * DSA_DIM : 0);
  static constexpr int OFF_SCL = OFF_VU + (KV8 ? VUR * VUB : 0);       // e4m3: float [RR][3][128]: of each token scale x the scores' factor, log2 and 1 / scale
  static constexpr int OFF_ROWS = OFF_SCL + (KV8 ? RR * 3 * NT * 4 : 0);      // int32 [RR][128]: pool row or -1
  static constexpr int OFF_MASK = OFF_ROWS + RR * NT * 4;            // uint32 [RR][4]: tokens that count
  static constexpr int OFF_RUNS = OFF_MASK + RR * 4 * 4;             // uint32 [4]: bit i: rows 16 i .. 16 i + 15 are consecutive, or none is held
  static constexpr int OFF_QMUL = OFF_RUNS + 16;                     // float [QM][64], by segment
  static constexpr int OFF_MX = OFF_QMUL + QM * RH * 4;              // float [2][4][64]: between the parts of a row
  static constexpr int OFF_SCAN = OFF_MX + 8 * RH * 4;               // int64 [28]; the share's first and last tile; its first query, and that one's tile and tiles
  static constexpr int OFF_BAR = OFF_SCAN + 32 * 8;
  static constexpr int NBAR = 2 * RR + 2 * KS + 2 * VR + 4 + 4 + (KV8 ? 1 + 2 * KU + 2 * VUR : 0);
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
  static_assert(SMEM_BYTES <= 232448, "shared memory exceeds the sm_100 limit");
  static_assert(WARPS <= 28, "scan");
  static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0 && OFF_P % 1024 == 0, "atoms of the swizzle");
  static_assert(OFF_KU % 128 == 0 && KUB % 128 == 0 && OFF_VU % 128 == 0, "TMA boxes");
  static_assert(OFF_SCL % 16 == 0 && OFF_ROWS % 16 == 0, "16-byte reads");
  static_assert(OFF_SCAN % 8 == 0 && OFF_BAR % 8 == 0, "64-bit words and barriers");
};
constexpr uint32_t O_COL = 0, S_COL = 256, TMEM_COLS = 512;

struct AttendArgs {
  const __nv_bfloat16* q;
  const uint8_t* pool;
  const float* kv_scales;
  const int32_t* page_table;
  const int32_t* q_offsets;
  const int32_t* q_vis;
  const int32_t* idx;
  __nv_bfloat16* out;
  float* lse;
  int32_t* desc;
  float* o_part;
  float* l_part;
  uint32_t* err;
  int max_pages, num_pages, page_shift, block_shift;
  int B, Q, H, topk, sinks, window;
  float scale_log2;
};

// pool rows by boxes of one row, for gathers, and of several consecutive ones
struct AttendMaps {
  CUtensorMap q;                                     // [Q * H][576], boxes of 64 dims x a CTA's heads
  CUtensorMap row;                                   // 64 dims (bf16) or 256 codes
  CUtensorMap run;                                   // bf16: 8 rows x 3 chunks of 64 dims; e4m3: 16 rows x 256 codes
  CUtensorMap row_hi;                                // e4m3: 320 codes, in words of four
  CUtensorMap run_hi;                                // bf16: 16 rows x 4 chunks; e4m3: 16 rows x 320 codes
};

// The list of a query with `vis` visible tokens, laid out in entries: the
// sinks, up to a multiple of 16, then the window from a multiple of 16 on, so
// that 16 entries lie in one page of 16 or more tokens.  Entries that the list
// does not hold are position -1.
struct List {
  int ns;           // sinks: entry j < ns is position j
  int ns_pad;
  int w0;           // first position of the window
  uint32_t n;       // entries: at most 30 more than tokens
  __device__ __forceinline__ int position(uint32_t j) const {
    const uint32_t pad = ns_pad;
    if (j < pad) return j < static_cast<uint32_t>(ns) ? static_cast<int>(j) : -1;
    const uint32_t p = (w0 & ~(RUN - 1)) + (j - pad);
    return j < n && p >= static_cast<uint32_t>(w0) ? static_cast<int>(p) : -1;
  }
};

// whether a sequence holds query q; the results of others stay as they were
__device__ __forceinline__ bool held(const AttendArgs& a, int q) {
  const int first = a.q_offsets[0], end = a.q_offsets[a.B];
  return (q >= first) & (q < end);
}

// tokens it attends to, of `seen` visible ones: those that its pages can hold
__device__ __forceinline__ int visible(const AttendArgs& a, bool mine, int seen) {
  const int v = mine ? max(0, seen) : 0;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_shift;
  return v < cap ? v : static_cast<int>(cap);
}

__device__ __forceinline__ List list_of(const AttendArgs& a, int vis) {
  List l;
  l.ns = min(a.sinks, vis);
  l.w0 = max(l.ns, vis - a.window);
  if (l.w0 == l.ns) l.ns = l.w0 = 0;                 // one range
  l.ns_pad = l.ns > 0x7FFFFFF0 ? l.ns : (l.ns + RUN - 1) & ~(RUN - 1);
  l.n = static_cast<uint32_t>(l.ns_pad) + (vis > l.w0 ? vis - (l.w0 & ~(RUN - 1)) : 0);
  return l;
}

// tiles of query q: at least one, which writes the result of an empty list
template <bool IDX>
__device__ __noinline__ int tiles_of(const AttendArgs& a, int q) {
  if constexpr (IDX) return (a.topk + NT - 1) / NT;
  const int seen = a.q_vis[q];                       // in flight beside the offsets
  return max(1u, (list_of(a, visible(a, held(a, q), seen)).n + NT - 1) / NT);
}

// Waits of a whole warp for the phase of the given parity, bounded by their
// number of tries: 2^22 of at most 200 ns and some 100 cycles each, about one second.
// A try suspends the warp for up to WAIT_NS, so that it leaves the issue slots to
// others: polled barriers took half of all slots.  WAIT_NS bounds how late an arrival
// from the peer CTA is seen.  A wait that gives up does so a second after the copies
// that were issued before it, so they have landed when its warp ends.
constexpr uint32_t WAIT_TRIES = 1u << 22, WAIT_NS = 200;
__device__ __forceinline__ bool try_wait_ns(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(WAIT_NS)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, uint32_t* err) {
#pragma unroll 1
  for (uint32_t it = 0; !__all_sync(0xffffffffu, try_wait_ns(bar, parity)); ++it) {
    if (it == WAIT_TRIES) {
      raise_error(err, DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// two of them, their answers under way together
__device__ __forceinline__ bool await_both(uint64_t* bar0, uint32_t parity0, uint64_t* bar1, uint32_t parity1,
                                           uint32_t* err) {
#pragma unroll 1
  for (uint32_t it = 0;; ++it) {
    const bool first = try_wait_ns(bar0, parity0), second = try_wait_ns(bar1, parity1);
    if (__all_sync(0xffffffffu, first && second)) return true;
    if (it == WAIT_TRIES) {
      raise_error(err, DEVERR_TIMEOUT);
      return false;
    }
  }
}

// a ring of N slots: the one in turn, and the parity of its use
template <int N>
struct Ring {
  uint32_t slot = 0, use = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      use ^= 1;
    }
  }
};

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// both CTAs' operands: the same offsets in each one's shared and tensor memory
__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrive on `bar` of both CTAs when every MMA issued so far is done
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Arrive on a barrier of the cluster (its address there) after this CTA's own
// shared-memory writes, which the fence before has made the tensor core's.  At
// the default scope: a release at cluster scope (mbar_arrive_remote) waits for
// every access under way, 1300 to 2000 cycles here.  That CTA scope is enough is an
// assumption: the other CTA's warp that waits for it reads none of the data, it issues
// MMAs, and this SM's tensor core reads this SM's shared memory, where the fence has
// put the writes.
// The lane that arrives leaves its branch by a __syncwarp: the tcgen05, cluster and
// named barrier instructions behind it are undefined for a warp that is not whole.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 16 bytes of shared memory
__device__ __forceinline__ uint4 lds16(const void* p) { return *static_cast<const uint4*>(p); }

// loads whose bytes count on a barrier of either CTA of the pair
__device__ __forceinline__ void gather4_pair(void* dst, const CUtensorMap* map, int x, uint4 r, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_3d_pair(void* dst, const CUtensorMap* map, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// four e4m3 codes -> four fp16, exactly.  Written in PTX: with the intrinsic of the
// pair type a warp took 800 cycles for its part of a raw unit, with this 479.
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  uint2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(w));
  return r;
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// larger of m and the magnitude bits of a bf16 pair's two values
__device__ __forceinline__ uint32_t mag2(uint32_t m, uint32_t w) {
  return max(max(m, (w << 16) & 0x7FFF0000u), w & 0x7FFF0000u);
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float s) {
  return f16x2_bits(__uint_as_float(w << 16) * s, __uint_as_float(w & 0xFFFF0000u) * s);
}

// 16 codes of a token, widened: pieces p and p + 1 of the 128-byte row dst, whose
// swizzle is sw; `flip` stores the second first
__device__ __forceinline__ void store_wide(uint8_t* dst, int p, int sw, int flip, uint4 c) {
  const uint2 w0 = widen4(c.x), w1 = widen4(c.y), w2 = widen4(c.z), w3 = widen4(c.w);
  const uint4 lo = make_uint4(w0.x, w0.y, w1.x, w1.y), hi = make_uint4(w2.x, w2.y, w3.x, w3.y);
  *reinterpret_cast<uint4*>(dst + (((p + flip) ^ sw) << 4)) = flip ? hi : lo;
  *reinterpret_cast<uint4*>(dst + (((p + 1 - flip) ^ sw) << 4)) = flip ? lo : hi;
}

// The query as fp16 in place, each head scaled so that its largest element lies
// in [2^14, 2^15); infinities and NaN stay what they are.  A warp takes
// an eighth of the heads, two at a time; 72 pieces of 8 dims a head.  A function of
// its own, since two places call it.
__device__ __noinline__ void scale_query(uint8_t* qs, float* qmul, int heads, int lw, int lane) {
#pragma unroll 1
  for (int h0 = heads * lw; h0 < heads * (lw + 1); h0 += 2) {
    uint4 v[2][3];
    auto piece = [&](int r, int k) {
      const int p = 32 * k + lane;
      return reinterpret_cast<uint4*>(qs + (p >> 3) * CH + r * 128 + (((p & 7) ^ (r & 7)) << 4));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int k = 0; k < 3; ++k) v[i][k] = k < 2 || lane < 8 ? *piece(h0 + i, k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k) m = mag2(mag2(mag2(mag2(m, v[i][k].x), v[i][k].y), v[i][k].z), v[i][k].w);
      m = __reduce_max_sync(0xffffffffu, m) >> 16;
      const int e = min(max(static_cast<int>(m >> 7), 14), 254);
      const float s = m == 0 || m >= 0x7F80u ? 1.f : __uint_as_float(static_cast<uint32_t>(min(254, 268 - e)) << 23);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k < 2 || lane < 8)
          *piece(h0 + i, k) = make_uint4(scale_pair(v[i][k].x, s), scale_pair(v[i][k].y, s), scale_pair(v[i][k].z, s),
                                         scale_pair(v[i][k].w, s));
      if (lane == 0) qmul[h0 + i] = __fdiv_rn(1.f, s);
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// first row of a run: of rows that the list does not hold, all before the pool
__device__ __forceinline__ int run_start(int row) { return row < 0 ? -RUN : row; }

template <bool KV8, bool IDX>
__global__ void __launch_bounds__(Plan<KV8>::THREADS, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ AttendMaps maps) {
  using L = Plan<KV8>;
  constexpr int THREADS = L::THREADS, KG = L::KG, KS = L::KS, KCH = L::KCH, VR = L::VR;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's atoms: 1024 bytes
  uint8_t* qs = smem + L::OFF_Q;
  uint8_t* ks = smem + L::OFF_K;
  uint8_t* vs = smem + L::OFF_V;
  uint8_t* ps = smem + L::OFF_P;
  float* scl = reinterpret_cast<float*>(smem + L::OFF_SCL);
  int* rows = reinterpret_cast<int*>(smem + L::OFF_ROWS);
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + L::OFF_MASK);
  uint32_t* runs = reinterpret_cast<uint32_t*>(smem + L::OFF_RUNS);
  float* qmul = reinterpret_cast<float*>(smem + L::OFF_QMUL);
  float* mx = reinterpret_cast<float*>(smem + L::OFF_MX);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + L::OFF_SCAN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  // "full" barriers of the MMAs' operands are the first CTA's, fed by both;
  // the MMAs arrive on both CTAs' "empty" ones
  uint64_t* r_full = bars;                 // [RR] rows of a tile are looked up
  uint64_t* r_empty = r_full + RR;
  uint64_t* k_full = r_empty + RR;         // [KS]
  uint64_t* k_empty = k_full + KS;
  uint64_t* v_full = k_empty + KS;         // [VR]
  uint64_t* v_empty = v_full + VR;
  uint64_t* s_full = v_empty + VR;         // [2] scores of a tile are in their slot
  uint64_t* s_empty = s_full + 2;          // [2] they are read
  uint64_t* p_full = s_empty + 2;          // P of a tile is in shared memory
  uint64_t* pv_done = p_full + 1;          // its value MMAs are done: P is free, O holds
  uint64_t* q_full = pv_done + 1;          // a segment's query is in shared memory
  uint64_t* q_empty = q_full + 1;          // its scores are done
  uint64_t* q_raw = q_empty + 1;           // e4m3: this CTA's part as bf16
  uint64_t* ku_full = q_raw + 1;           // e4m3: [2] units of key codes
  uint64_t* ku_empty = ku_full + KU;
  uint64_t* vu_full = ku_empty + KU;       // e4m3: [2] units of value codes
  uint64_t* vu_empty = vu_full + VUR;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
  int* held_rows = reinterpret_cast<int*>(tmem_holder + 1);   // [2] the sequences' first query, and one past the last

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int HC = a.H >> 1;                           // this CTA's heads: 64 or 32
  const int live_smx = a.H == 128 ? SMX : SMX / 2;   // warps whose rows hold heads
  pdl_trigger();
  if (tid == 32) {
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.row);
    tma_prefetch_desc(&maps.run);
    if (KV8) {
      tma_prefetch_desc(&maps.row_hi);
      tma_prefetch_desc(&maps.run_hi);
    }
  }

  if (tid < L::NBAR) {
    // arrivals a phase: one, but for these
    const int i = tid;
    const int full = KV8 ? 2 * GROUP : 1;            // widened operands: a warp each
    int n = 1;
    if (i >= RR && i < 2 * RR) n = 2 + live_smx;
    if (i >= k_full - bars && i < k_empty - bars) n = KV8 ? 2 * GROUP : 1;
    if (i >= v_full - bars && i < v_empty - bars) n = full;
    if (i >= s_empty - bars && i <= p_full - bars) n = 2 * live_smx;
    if (i == q_full - bars) n = KV8 ? 4 * GROUP : 1;
    if (KV8 && i >= ku_empty - bars && i < vu_full - bars) n = 2 * GROUP;
    if (KV8 && i >= vu_empty - bars) n = GROUP;
    mbar_init(bars + i, n);
    mbar_fence_init();
  }
  if (warp == 0) {
    __syncwarp();                                    // the allocation wants its warp whole
    tmem_alloc_pair(tmem_holder, TMEM_COLS);
  }
  // So far nothing was read or written that another kernel touches.  What is read from
  // here on may have been written beside the lines above, by an append or a selector,
  // so these are plain loads, not those for data that stays constant while a kernel lives.
  pdl_wait();

  // This pair's share [t0, t1) of all tiles: a thread sums the tiles of some
  // consecutive queries, the block scans the sums.  Where there is enough of
  // them a query counts START tiles more, about what it costs to begin one.
  const int per = (a.Q + THREADS - 1) / THREADS;
  const int qa = min(a.Q, tid * per), qb = min(a.Q, qa + per);
  int64_t sum = 0;
#pragma unroll 1
  for (int q = qa; q < qb; ++q) sum += tiles_of<IDX>(a, q);
  int64_t incl = sum;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  if (tid < 2) {
    scan[28 + tid] = 0;
    held_rows[tid] = a.q_offsets[tid * a.B];
  }
  __syncthreads();
  int64_t before = lane < THREADS / 32 ? scan[lane] : 0;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  const int64_t total = __shfl_sync(0xffffffffu, before, 31);
  const int64_t base = __shfl_sync(0xffffffffu, before, warp) - scan[warp] + incl - sum;
  const int start = total >= 4 * pairs ? START : 0;
  const uint32_t np = total < pairs ? static_cast<uint32_t>(total) : pairs;   // pairs that get work
  const int64_t cost = total + static_cast<int64_t>(start) * a.Q;
  const int64_t each = cost >> 32 ? cost / np : static_cast<uint32_t>(cost) / np;
  const uint32_t over = static_cast<uint32_t>(cost - each * np);
  // where the shares of this pair and of the next one begin
#pragma unroll 1
  for (uint32_t i = 0; i < 2; ++i) {
    const uint32_t p = min(pair + i, np);
    const int64_t c = p == np ? cost : each * p + min(p, over);
    if (p == np) {
      if (tid == 0) scan[28 + i] = total;
    } else {
      int64_t at = base;
      const int64_t at_cost = base + static_cast<int64_t>(start) * qa;
      if (c >= at_cost && c < at_cost + sum + static_cast<int64_t>(start) * (qb - qa)) {
        int64_t left = c - at_cost;
        int q = qa, n;
#pragma unroll 1
        for (; left >= start + (n = tiles_of<IDX>(a, q)); ++q) {
          left -= start + n;
          at += n;
        }
        const int64_t off = left > start ? left - start : 0;
        scan[28 + i] = at + off;
        if (i == 0) {
          scan[30] = q;
          scan[31] = off | static_cast<int64_t>(n) << 32;
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  __syncthreads();                                   // the share is known
  // its first query's loads, while the other CTA arrives
  int seen0 = 0, seq0 = 0;
  if (warp == 3 && scan[29] > scan[28]) {
    seen0 = a.q_vis[scan[30]];
    seq0 = seq_of_query_warp(a.q_offsets, a.B, static_cast<int>(scan[30]), lane);
  }
  __syncwarp();
  cluster_wait();                                    // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int q0 = static_cast<int>(scan[30]);
  const int off0 = static_cast<int>(scan[31]);
  const int ntile = static_cast<int>(scan[29] - scan[28]);
  if (half == 0 && tid < 2 && ntile == 0) a.desc[2 * pair + tid] = -1;

  // the tiles of the share's first query are known already
  auto tiles = [&](int q) {
    if constexpr (!IDX)
      if (q == q0) return static_cast<int>(scan[31] >> 32);
    return tiles_of<IDX>(a, q);
  };
  // the first CTA's barrier of the same name
  auto leader = [&](uint64_t* bar) { return map_to_rank(smem_u32(bar), 0); };
  // a warp's part of an operand is written: tell the MMA issuer
  auto hand_over = [&](uint64_t* bar) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(leader(bar));
    __syncwarp();
  };
  // slot of a tile's key group j, and the parity of its use: slots 0 and 1 of an
  // e4m3 tile are used twice
  auto key_slot = [](int j) { return KV8 ? (j == 4 ? 2 : j & 1) : j; };
  auto key_use = [](int j, uint32_t g) { return KV8 && j < 4 ? static_cast<uint32_t>(j >> 1) : g & 1; };
  // the query of a segment, once the scores of the one before are done
  auto load_query = [&](int q, uint32_t seg, bool lead) {
    if (seg > 0 && !await(q_empty, (seg - 1) & 1, a.err)) return false;
    if (lead) {
      const uint32_t bytes = static_cast<uint32_t>(KC * 128 * HC);
      const uint32_t bar = KV8 ? smem_u32(q_raw) : leader(q_full);
      if (KV8) mbar_arrive_expect_tx(q_raw, bytes);
      else if (half == 0) mbar_arrive_expect_tx(q_full, 2 * bytes);
#pragma unroll 1
      for (int c = 0; c < KC; ++c) load_2d_pair(qs + c * CH, &maps.q, 64 * c, q * a.H + half * HC, bar);
    }
    __syncwarp();
    return true;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ score MMAs
    // The warp walks together, so that descriptors stay in uniform registers,
    // and one elected lane issues.
    constexpr uint32_t fmt = KV8 ? 0u /*F16*/ : 1u /*BF16*/;
    constexpr uint32_t idesc_s = umma_idesc(fmt, 128, NT);
    const uint64_t dq = umma_desc_sw128(smem_u32(qs), 1024, 16);
    const uint64_t dk = umma_desc_sw128(smem_u32(ks), KV8 ? 1024 : 1024 * KCH, 16);
    const bool lead = elect_one();
    bool ok = true;
    int q = q0, off = off0, left = half == 0 ? ntile : 0;
    uint32_t g = 0;                              // tiles so far
#pragma unroll 1
    for (uint32_t seg = 0; left > 0 && ok; ++seg, ++q, off = 0) {
      const int n = min(tiles(q) - off, left);
      left -= n;
      if (!(ok = await(q_full, seg & 1, a.err))) break;
#pragma unroll 1
      for (int u = 0; u < n && ok; ++u, ++g) {
        const uint32_t d = tmem + S_COL + (g & 1) * NH;
        if (!(ok = await(&s_empty[g & 1], ((g >> 1) & 1) ^ 1, a.err))) break;
#pragma unroll 1
        for (int j = 0; j < KG; ++j) {
          const int slot = key_slot(j), nc = KV8 && j == 4 ? 1 : KCH;
          if (!(ok = await(&k_full[slot], key_use(j, g), a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
              const uint64_t dqc = dq + (KCH * j + c) * (CH >> 4), dkc = dk + (KCH * slot * CH + c * (KV8 ? CH : 1024)) / 16;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_pair(d, dqc + k * 2, dkc + k * 2, idesc_s, j > 0 || c > 0 || k > 0 ? 1u : 0u);
            }
            mma_commit_pair(&k_empty[slot]);
            if (j == KG - 1) {
              mma_commit_pair(&s_full[g & 1]);
              if (u == n - 1) mma_commit_pair(q_empty);
            }
          }
          __syncwarp();
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ queries, keys
    // A load takes about 45 cycles to issue whatever its size, so its box is as
    // large as consecutive rows allow.  Lane 4 i + t: rows 4 t .. 4 t + 3 of the
    // 16 rows i, or of a run lane 4 i (bf16: and 4 i + 2) for all.  A slot of the
    // bf16 keys holds 8 rows x 3 chunks after another.
    const bool lead = elect_one();
    bool ok = true;
    int q = q0, off = off0, left = ntile;
    uint32_t g = 0;
    if (ntile > 0) load_query(q, 0, lead);
#pragma unroll 1
    for (uint32_t seg = 0; left > 0 && ok; ++seg, ++q, off = 0) {
      const int n = min(tiles(q) - off, left);
      left -= n;
#pragma unroll 1
      for (int u = 0; u < n && ok; ++u, ++g) {
        const uint32_t slot = g % RR;
        if (!(ok = await(&r_full[slot], (g / RR) & 1, a.err))) break;
        const bool run = KV8 ? runs[slot] >> (half * (NH / 16) + (lane >> 2 & 3)) & 1u
                             : runs[slot] >> (8 + half * (NH / 8) + (lane >> 1 & 7)) & 1u;
        const uint4 r = lds16(rows + slot * NT + half * NH + 4 * (lane & 15));
        const int r0 = run_start(static_cast<int>(r.x));
        const int i = lane >> 2, t = lane & 3;
#pragma unroll 1
        for (int j = 0; j < (KV8 ? KU : 3); ++j) {
          uint64_t* full = KV8 ? &ku_full[j] : &k_full[j];
          if (!(ok = await(KV8 ? &ku_empty[j] : &k_empty[j], (g & 1) ^ 1, a.err))) break;
          if constexpr (KV8) {
            const int pitch = j == 0 ? 256 : 320;
            uint8_t* dst = smem + L::OFF_KU + j * KUB + lane * 4 * pitch;
            if (lead) mbar_arrive_expect_tx(full, NH * pitch);
            __syncwarp();
            if (lane < 16 && !run)
              gather4_pair(dst, j == 0 ? &maps.row : &maps.row_hi, 64 * j, r, smem_u32(full));
            __syncwarp();
            if (lane < 16 && run && t == 0)
              load_2d_pair(dst, j == 0 ? &maps.run : &maps.run_hi, 64 * j, r0, smem_u32(full));
          } else {
            const uint32_t bar = leader(full);
            uint8_t* dst = ks + j * KCH * CH + (i * 2 + (t >> 1)) * KCH * 1024 + (t & 1) * 512;
            if (half == 0 && lead) mbar_arrive_expect_tx(full, 2 * KCH * CH);
            __syncwarp();
            if (lane < 16 && !run) {
#pragma unroll 1
              for (int c = 0; c < KCH; ++c) gather4_pair(dst + c * 1024, &maps.row, 64 * (KCH * j + c), r, bar);
            }
            __syncwarp();
            if (lane < 16 && run && (t & 1) == 0) load_3d_pair(dst, &maps.run, r0, KCH * j, bar);
          }
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&r_empty[slot]);
        __syncwarp();
        if (u == 0 && seg > 0 && ok) ok = load_query(q, seg, lead);   // its keys are on their way
      }
    }
    // the MMAs have read every key, so no load is under way
    if constexpr (!KV8) {
#pragma unroll 1
      for (int j = 0; j < KG && ok && ntile > 0; ++j) ok = await(&k_empty[j], (ntile - 1) & 1, a.err);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ values
    // A unit is two times 16 rows.  e4m3: lane 4 i + t as above; bf16: lane
    // 16 i + 4 c + t dims 64 c .. 64 c + 63 of rows 4 t .. 4 t + 3, or lane 16 i
    // all of a run.
    const bool lead = elect_one();
    bool ok = true;
    Ring<KV8 ? VUR : VR> ur;
#pragma unroll 1
    for (int g = 0; g < ntile && ok; ++g) {
      const uint32_t slot = g % RR;
      if (!(ok = await(&r_full[slot], (g / RR) & 1, a.err))) break;
      const int i = KV8 ? lane >> 2 & 1 : lane >> 4;
      const uint32_t run_bits = runs[slot] >> i;
      const int* rr = rows + slot * NT + i * RUN + 4 * (lane & 3);
#pragma unroll 1
      for (int c = 0; c < VS; ++c, rr += VT) {
        const uint4 r = lds16(rr);
        const bool run = (run_bits >> (2 * c)) & 1u;
        const int r0 = run_start(static_cast<int>(r.x));
        uint64_t* full = KV8 ? &vu_full[ur.slot] : &v_full[ur.slot];
        if (!(ok = await(KV8 ? &vu_empty[ur.slot] : &v_empty[ur.slot], ur.use ^ 1, a.err))) break;
        if constexpr (KV8) {
          uint8_t* dst = smem + L::OFF_VU + ur.slot * VUB + lane * 1024;
          if (lead) mbar_arrive_expect_tx(full, VUB);
          __syncwarp();
          if (lane < 8 && !run) gather4_pair(dst, &maps.row, 256 * half, r, smem_u32(full));
          __syncwarp();
          if (lane < 8 && run && (lane & 3) == 0) load_2d_pair(dst, &maps.run, 256 * half, r0, smem_u32(full));
        } else {
          const uint32_t bar = leader(full);
          const int d = lane >> 2 & 3;
          uint8_t* dst = vs + ur.slot * VSLOT + i * VSTEP + d * VCH + (lane & 3) * 512;
          if (half == 0 && lead) mbar_arrive_expect_tx(full, 2 * VSLOT);
          __syncwarp();
          if (!run) gather4_pair(dst, &maps.row, 256 * half + 64 * d, r, bar);
          __syncwarp();
          if (run && (lane & 15) == 0) load_3d_pair(dst, &maps.run_hi, r0, 4 * half, bar);
        }
        __syncwarp();
        ur.next();
      }
      if (lane == 0) mbar_arrive(&r_empty[slot]);
      __syncwarp();
    }
    if constexpr (!KV8) {
#pragma unroll 1
      for (int i = 0; i < VR && ok && ntile > 0; ++i) {
        ok = await(&v_empty[ur.slot], ur.use ^ 1, a.err);
        ur.next();
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ row look-up
    // Three dependent loads a token (selected position, page, scale), of which
    // each step of the loop issues one for each of three tiles.
    bool ok = true, bad = false;
    int q = q0 - 1, off = 0, n = 0, left = ntile, u = 0;
    int vis = 0;
    List ls = {};
    int pos[4], at[4], pg[4], row[4];                // tile i; tile i - 1; tile i - 2
    float s[4];
    const int32_t *pages = a.page_table, *pages1 = pages;
    int vis1 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) pos[k] = at[k] = pg[k] = row[k] = -1;
#pragma unroll 1
    for (int i = 0; i < ntile + 3 && ok; ++i) {
      if (i >= 3) {
        // tile i - 3: hand it over
        const uint32_t g = i - 3, slot = g % RR;
        if (!(ok = await(&r_empty[slot], ((g / RR) & 1) ^ 1, a.err))) break;
        if constexpr (KV8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (row[k] >= 0 && !(s[k] >= 0x1p-40f && s[k] <= 0x1p40f)) {
              row[k] = -1;
              bad = true;
            }
            const float st = row[k] < 0 ? 1.f : s[k];
            float* sc = scl + slot * 3 * NT + 32 * k + lane;
            sc[0] = st * a.scale_log2;
            sc[NT] = log2f(st);
            sc[2 * NT] = __fdiv_rn(1.f, st);
          }
        }
        uint32_t run = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          rows[slot * NT + 32 * k + lane] = row[k];
          const uint32_t m = __ballot_sync(0xffffffffu, row[k] >= 0);
          if (lane == 0) mask[slot * 4 + k] = m;
          const int first = __shfl_sync(0xffffffffu, row[k], lane & 16);
          const uint32_t c =
              __ballot_sync(0xffffffffu, first >= 0 ? row[k] == first + (lane & 15) : row[k] < 0);
          run |= ((c & 0xFFFFu) == 0xFFFFu ? 1u : 0u) << (2 * k) | (c >> 16 == 0xFFFFu ? 2u : 0u) << (2 * k);
          if constexpr (!KV8) {
            // bf16 keys: runs of 8 rows, in the upper bits
            const int first8 = __shfl_sync(0xffffffffu, row[k], lane & 24);
            const uint32_t c8 = __ballot_sync(0xffffffffu, first8 >= 0 ? row[k] == first8 + (lane & 7) : row[k] < 0);
#pragma unroll
            for (int b = 0; b < 4; ++b) run |= ((c8 >> (8 * b) & 0xFFu) == 0xFFu ? 1u : 0u) << (8 + 4 * k + b);
          }
        }
        if (lane == 0) runs[slot] = run;
        __syncwarp();
        if (lane == 0) mbar_arrive(&r_full[slot]);
        __syncwarp();
      }
      // tile i - 2: its pages are here; tile i - 1: its positions are here
      // (before the first and behind the last tile these are -1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        row[k] = -1;
        if (pg[k] >= 0 && pg[k] < a.num_pages) row[k] = (pg[k] << a.page_shift) + (at[k] & ((1 << a.page_shift) - 1));
        bad |= at[k] >= 0 && row[k] < 0;
        if constexpr (KV8) s[k] = row[k] >= 0 ? a.kv_scales[row[k] >> a.block_shift] : 1.f;
        // The row on its way to L2, half a row a CTA: it is loaded about two tiles
        // from now, which a load from DRAM would not quite fit into.
        if (row[k] >= 0) {
          constexpr int ROW = DSA_DIM * (KV8 ? 1 : 2), LINES = (ROW / 2 + 127) / 128;
          const uint8_t* at_row = a.pool + static_cast<size_t>(row[k]) * ROW + half * (ROW / 2);
#pragma unroll
          for (int l = 0; l < LINES; ++l) prefetch_l2(at_row + l * 128);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        at[k] = pos[k] >= 0 && pos[k] < vis1 ? pos[k] : -1;
        bad |= at[k] != pos[k] && pos[k] != -1 && vis1 >= 0;
        pg[k] = at[k] >= 0 ? pages1[at[k] >> a.page_shift] : -1;
      }
      if (i < ntile && u == n) {
        ++q;
        off = i == 0 ? off0 : 0;
        n = min(tiles(q) - off, left);
        left -= n;
        u = 0;
        const int seen = i == 0 ? seen0 : a.q_vis[q];   // in flight beside the search
        const int seq = i == 0 ? seq0 : seq_of_query_warp(a.q_offsets, a.B, q, lane);
        const bool mine = q >= held_rows[0] && q < held_rows[1];
        pages = a.page_table + static_cast<size_t>(seq) * a.max_pages;
        vis = visible(a, mine, seen);
        ls = list_of(a, vis);
        if (!mine) vis = -1;                         // nothing is read, and no index is a fault
        else bad |= seen > vis;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t j = static_cast<uint32_t>(off + u) * NT + 32 * k + lane;
        pos[k] = -1;
        if (i < ntile) {
          if constexpr (IDX) {
            if (j < static_cast<uint32_t>(a.topk)) pos[k] = a.idx[static_cast<size_t>(q) * a.topk + j];
          } else {
            pos[k] = ls.position(j);
          }
        }
      }
      pages1 = pages;
      vis1 = vis;
      ++u;
    }
    if (bad) raise_error(a.err, DEVERR_BOUNDS);
    __syncwarp();
  } else if (warp < SMX0 + SMX) {
    // ------------------------------------------------------------ softmax, output
    // thread: accumulator row r, the tile's tokens 64 hh + 32 cg .. + 31, and
    // value dims 256 hh + 128 cg .. + 127; part = 2 hh + cg
    if constexpr (KV8) asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    const int quarter = warp & 3, hh = quarter >> 1, cg = (warp - SMX0) >> 2;
    const int r = (quarter & 1) * 32 + lane;
    const int h = half * HC + r;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t row_bar = 1 + (quarter & 1);      // the four warps of the same rows
    constexpr float RAISE = KV8 ? 7.f : 0.f;         // P = 2^(z - m + RAISE)
    bool ok = true;
    int q = q0, off = off0, left = r < HC ? ntile : 0;
    uint32_t g = 0;
    int head_q = -1, tail_q = -1;                    // queries this pair holds a part of
#pragma unroll 1
    for (uint32_t seg = 0; left > 0; ++seg, ++q, off = 0) {
      const int nt = tiles(q);
      const int n = min(nt - off, left);
      left -= n;
      float qm = 1.f, m_use = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int u = 0; u < n; ++u, ++g) {
        const uint32_t sb = g & 1, slot = g % RR;
        if (ok) ok = await_both(&r_full[slot], (g / RR) & 1, &s_full[sb], (g >> 1) & 1, a.err);
        tc_fence_after();
        const uint32_t live = mask[slot * 4 + 2 * hh + cg];
        float z[32];
        tmem_ld32(lane_base + S_COL + sb * NH + cg * 32, z);
        // the scores are there, so the query's factors are
        if (KV8 && u == 0) qm = qmul[(seg % QM) * RH + r];
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(leader(&s_empty[sb]));
        __syncwarp();
        float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const float* sc = scl + slot * 3 * NT + hh * NH + cg * 32;
        if constexpr (KV8) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 k = *reinterpret_cast<const float4*>(sc + j);
            const float4 e = *reinterpret_cast<const float4*>(sc + NT + j);
            z[j] = fmaf(z[j] * k.x, qm, e.x);
            z[j + 1] = fmaf(z[j + 1] * k.y, qm, e.y);
            z[j + 2] = fmaf(z[j + 2] * k.z, qm, e.z);
            z[j + 3] = fmaf(z[j + 3] * k.w, qm, e.w);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] *= a.scale_log2;
        }
        if (live != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = ((live >> j) & 1u) ? z[j] : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) mt[j & 3] = fmaxf(mt[j & 3], z[j]);
        float mtile = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
        float* mxs = mx + (g & 1) * 4 * RH + r;
        mxs[(2 * hh + cg) * RH] = mtile;
        named_barrier(row_bar, 128);
        mtile = fmaxf(fmaxf(mxs[0], mxs[RH]), fmaxf(mxs[2 * RH], mxs[3 * RH]));
        // the maximum that P refers to moves only when it falls 8 behind, so O is
        // seldom rescaled; with RAISE P reaches 2^15, which fp16 holds
        float alpha = 1.f;
        bool resc = false;
        if (mtile > m_use + 8.f) {
          if (m_use != -INFINITY) {
            alpha = fast_exp2(m_use - mtile);
            resc = true;
          }
          m_use = mtile;
        }
        const float m_eff = m_use == -INFINITY ? 0.f : m_use - RAISE;
        float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = fast_exp2(z[j] - m_eff);
        if constexpr (KV8) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(sc + 2 * NT + j);
            sums[0] = fmaf(z[j], f.x, sums[0]);
            sums[1] = fmaf(z[j + 1], f.y, sums[1]);
            sums[2] = fmaf(z[j + 2], f.z, sums[2]);
            sums[3] = fmaf(z[j + 3], f.w, sums[3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) sums[j & 3] += z[j];
        }
        l = fmaf(l, alpha, (sums[0] + sums[1]) + (sums[2] + sums[3]));
        // the value MMAs of the tile before have read P and written O
        if (ok && g > 0) ok = await(pv_done, (g - 1) & 1, a.err);
        uint8_t* pr = ps + hh * CH + r * 128;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* zj = z + 8 * j;
          const uint4 w = KV8 ? make_uint4(f16x2_bits(zj[0], zj[1]), f16x2_bits(zj[2], zj[3]), f16x2_bits(zj[4], zj[5]),
                                           f16x2_bits(zj[6], zj[7]))
                              : make_uint4(bf16x2_bits(zj[0], zj[1]), bf16x2_bits(zj[2], zj[3]),
                                           bf16x2_bits(zj[4], zj[5]), bf16x2_bits(zj[6], zj[7]));
          *reinterpret_cast<uint4*>(pr + (((4 * cg + j) ^ (r & 7)) << 4)) = w;
        }
        if (__any_sync(0xffffffffu, resc)) {
          __syncwarp();
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            tmem_ld32(lane_base + O_COL + cg * 128 + c * 32, z);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] *= alpha;
            tmem_st32(lane_base + O_COL + cg * 128 + c * 32, z);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        hand_over(p_full);
        if (lane == 0) mbar_arrive(&r_empty[slot]);  // only now: the stores have waited for the loads
        __syncwarp();
      }
      // ---- the segment's result: the query's own, or a part of it
      float* mxs = mx + (g & 1) * 4 * RH + r;        // free: the tile before last used it
      mxs[(2 * hh + cg) * RH] = l;
      named_barrier(row_bar, 128);
      l = (mxs[0] + mxs[RH]) + (mxs[2 * RH] + mxs[3 * RH]);
      named_barrier(row_bar, 128);
      if (ok) ok = await(pv_done, (g - 1) & 1, a.err);
      tc_fence_after();
      const bool whole = n == nt;
      const bool head = off == 0;
      const int part = 2 * pair + (head ? 1 : 0);
      const bool mine = q >= held_rows[0] && q < held_rows[1];
      if (!whole && mine) (head ? head_q : tail_q) = q;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;   // NaN stays NaN
      const bool none = l == 0.f;
      // A part goes out as [dim / 4][head][4 dims], so that the lanes of a warp
      // write next to one another; a result by way of half of its rows of P (the
      // four warps of the same rows meet again before one writes P there), 64
      // bytes of eight heads a store.
      const int d0 = 256 * hh + 128 * cg;
      uint8_t* stage = ps + hh * CH + (quarter & 1) * 4096 + cg * 2048;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        tmem_ld32(lane_base + O_COL + cg * 128 + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i] * inv;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4)) =
                make_uint4(bf16x2_bits(o[8 * i], o[8 * i + 1]), bf16x2_bits(o[8 * i + 2], o[8 * i + 3]),
                           bf16x2_bits(o[8 * i + 4], o[8 * i + 5]), bf16x2_bits(o[8 * i + 6], o[8 * i + 7]));
          __syncwarp();
          const int piece = lane & 3;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int hr = 8 * i + (lane >> 2);
            const uint4 w = lds16(stage + hr * 64 + ((piece ^ (hr >> 1 & 3)) << 4));
            const size_t row = static_cast<size_t>(q) * a.H + half * HC + (quarter & 1) * 32 + hr;
            if (mine) *reinterpret_cast<uint4*>(a.out + row * DSA_DIM_V + d0 + 32 * c + 8 * piece) = w;
          }
          __syncwarp();
        } else {
          float4* dst = reinterpret_cast<float4*>(a.o_part) +
                        (static_cast<size_t>(part) * (DSA_DIM_V / 4) + (d0 + 32 * c) / 4) * a.H + h;
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i * a.H] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (hh == 0 && cg == 0 && mine)
        (whole ? a.lse + static_cast<size_t>(q) * a.H + h : a.l_part + static_cast<size_t>(part) * a.H + h)[0] =
            none ? -INFINITY : (m_use - RAISE + log2f(l)) * 0.69314718055994531f;
      tc_fence_before();                             // O was read before the next segment writes it
    }
    if (half == 0 && warp == SMX0 && lane == 0 && ntile > 0) {
      a.desc[2 * pair] = tail_q;
      a.desc[2 * pair + 1] = head_q;
    }
    __syncwarp();
  } else if (warp >= SMX0 + SMX + (KV8 ? 3 * GROUP : 0)) {
    // ------------------------------------------------------------ value MMAs
    // e4m3: the seven warp groups start with 72 registers a thread, of which the
    // softmax needs more, the widening and this group, one warp of which works, less:
    // 72 + 2 x 96 + 3 x 64 + 48 = 7 x 72
    if constexpr (KV8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    constexpr uint32_t idesc_pv = umma_idesc(KV8 ? 0u : 1u, 128, 256, 0, 1);
    const uint64_t dp = umma_desc_sw128(smem_u32(ps), 1024, 16);
    const uint64_t dv = umma_desc_sw128_mn(smem_u32(vs), VCH, 1024);
    const bool lead = elect_one();
    bool ok = true;
    int q = q0, off = off0, left = half == 0 && warp == SMX0 + SMX + (KV8 ? 3 * GROUP : 0) ? ntile : 0;
    uint32_t g = 0;
    Ring<VR> vr;
#pragma unroll 1
    for (; left > 0 && ok; ++q, off = 0) {
      const int n = min(tiles(q) - off, left);
      left -= n;
#pragma unroll 1
      for (int u = 0; u < n && ok; ++u, ++g) {
        if (!(ok = await(p_full, g & 1, a.err))) break;
#pragma unroll 1
        for (int i = 0; i < VS; ++i) {
          if (!(ok = await(&v_full[vr.slot], vr.use, a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < VT / 16; ++k) {
              const uint64_t dpi = dp + (i >> 1) * (CH >> 4) + (i & 1) * 4 + k * 2;
              const uint64_t dvi = dv + vr.slot * (VSLOT >> 4) + k * (VSTEP >> 4);
              const uint32_t acc = u > 0 || i > 0 || k > 0 ? 1u : 0u;
              mma_f16_pair(tmem + O_COL, dpi, dvi, idesc_pv, acc);
              mma_f16_pair(tmem + O_COL + 128, dpi, dvi + (2 * VCH >> 4), idesc_pv, acc);
            }
            mma_commit_pair(&v_empty[vr.slot]);
            if (i == VS - 1) mma_commit_pair(pv_done);
          }
          __syncwarp();
          vr.next();
        }
      }
    }
  } else if (KV8 && warp < SMX0 + SMX + 2 * GROUP) {
    // ------------------------------------------------------------ e4m3: keys widened, queries scaled
    // Two chunks at a time, the first and third pair of them by one group of four
    // warps, the second and fourth by another; the positions by the first.  thread:
    // 16 codes of four tokens.  Lanes of odd chunks store their two pieces in the
    // other order, so that the eight lanes of a store lie in different banks.
    if constexpr (KV8) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int lw = warp - (SMX0 + SMX), team = lw / GROUP;
    const int lt = (lw % GROUP) * 32 + lane;
    const int pc = lt & 7, r0 = lt >> 3, flip = pc >> 2, rp = lt >> 2;
    bool ok = true;
    int off = off0, left = ntile, n = 0, u = 0, q = q0;
    uint32_t seg = 0;
    auto query = [&]() {
      if (!(ok = ok && await(q_raw, seg & 1, a.err))) return;
      scale_query(qs, qmul + (seg % QM) * RH, HC >> 3, lw, lane);
      hand_over(q_full);
    };
    uint8_t* const dst = ks + team * 2 * CH + flip * CH + r0 * 128;
#pragma unroll 1
    for (int g = 0; g < ntile && ok; ++g) {
      if (u == n) {
        if (g > 0) {
          ++q;
          ++seg;
          off = 0;
        }
        n = min(tiles(q) - off, left);
        left -= n;
        u = 0;
        if (g == 0) query();                         // while its rows are looked up
      }
      const uint8_t* raw = smem + L::OFF_KU;
      uint4 v[4];
#pragma unroll 1
      for (int d = 0; d < 2; ++d) {
        const int pitch = 256 + 64 * d;
        const uint8_t* src = raw + d * KUB + r0 * pitch + team * 128 + pc * 16;
        const bool free = mbar_test_wait(&k_empty[team], d ^ 1);
        if (u == 0 && g > 0 && d == 1) query();      // both slots are full: their scores wait for the query
        if (!(ok = ok && await(&ku_full[d], g & 1, a.err))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lds16(src + i * 16 * pitch);
        if (!(ok = __all_sync(0xffffffffu, free) || await(&k_empty[team], d ^ 1, a.err))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) store_wide(dst + i * 16 * 128, 2 * (pc & 3), r0 & 7, flip, v[i]);
        hand_over(&k_full[team]);
        if (team == 0 && d == 1) {
          if (!(ok = await(&k_empty[2], (g & 1) ^ 1, a.err))) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) v[i] = lds16(raw + KUB + (rp + 32 * i) * 320 + 256 + (lt & 3) * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            store_wide(ks + 4 * CH + (rp + 32 * i) * 128, 2 * (lt & 3), rp & 7, 0, v[i]);
          hand_over(&k_full[2]);
        }
        if (lane == 0) mbar_arrive(&ku_empty[d]);    // only now: the stores have waited for the loads
        __syncwarp();
      }
      ++u;
    }
    // the MMAs have read every key
    if (ok && ntile > 0)
      ok = await(&k_empty[0], 1, a.err) && await(&k_empty[1], 1, a.err) && await(&k_empty[2], (ntile - 1) & 1, a.err);
  } else if (KV8) {
    // ------------------------------------------------------------ e4m3: values widened
    // A unit at a time.  thread: 16 codes of four tokens, as above.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int lt = (warp - (SMX0 + SMX + 2 * GROUP)) * 32 + lane;
    const int pc = lt & 15, r0 = lt >> 4, flip = (pc >> 2) & 1;
    bool ok = true;
    Ring<VR> vr;
    Ring<VUR> ur;
#pragma unroll 1
    for (int c = 0; c < ntile * VS && ok; ++c) {
      const bool free = mbar_test_wait(&v_empty[vr.slot], vr.use ^ 1);
      if (!(ok = await(&vu_full[ur.slot], ur.use, a.err))) break;
      const uint8_t* src = smem + L::OFF_VU + ur.slot * VUB + lt * 16;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lds16(src + i * 8 * 256);
      if (!(ok = __all_sync(0xffffffffu, free) || await(&v_empty[vr.slot], vr.use ^ 1, a.err))) break;
      uint8_t* dst = vs + vr.slot * VSLOT + (pc >> 2) * VCH + r0 * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) store_wide(dst + (i >> 1) * VSTEP + (i & 1) * 1024, 2 * (pc & 3), r0 & 7, flip, v[i]);
      hand_over(&v_full[vr.slot]);
      if (lane == 0) mbar_arrive(&vu_empty[ur.slot]);
      __syncwarp();
      vr.next();
      ur.next();
    }
    // the MMAs have read every value
#pragma unroll 1
    for (int i = 0; i < VR && ok && ntile > 0; ++i) {
      ok = await(&v_empty[vr.slot], vr.use ^ 1, a.err);
      vr.next();
    }
  }

  tc_fence_before();
  __syncwarp();
  cluster_sync();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}


// Merge of the parts of queries whose tiles lie on several pairs: pair p holds
// the first part of query desc[2p + 1] in part 2p + 1, the pairs after it the
// others in parts 2(p + i), where desc[2(p + i)] is that query again.
//   LSE = ln sum_i exp(LSE_i),  O = sum_i exp(LSE_i - LSE) O_i.
// The parts lie as [dim / 4][head][4 dims].  grid (pairs, H / 32, 4): 32 heads,
// a lane each, and 128 dims a CTA, 16 a warp; the result turns in shared memory.
// Bound by latency: the loads of several parts go out together, whether there are
// that many or not (one user's step over 2048 selected tokens 28.7 -> 27.4 us).
// Most CTAs find nothing to merge and end.  A grid that is resident at once and
// shares out what there is took 5 us more; a grid over the queries, 32 dims a CTA,
// where they are few: dense 4 x 128K 195 -> 194 us, one user 18.5 -> 19.3 us.
constexpr int MT = 256, MAX_PAIRS = 74;
__global__ void __launch_bounds__(MT, 4) attend_merge_kernel(const int32_t* desc, const float* o_part,
                                                             const float* l_part, int H, __nv_bfloat16* out,
                                                             float* lse) {
  __shared__ uint4 turn[32][17];
  __shared__ int tails[MAX_PAIRS], heads[MAX_PAIRS];
  pdl_trigger();
  pdl_wait();
  const int p = blockIdx.x, pairs = gridDim.x;
  if (threadIdx.x < pairs) {
    const int2 d = reinterpret_cast<const int2*>(desc)[threadIdx.x];
    tails[threadIdx.x] = d.x;
    heads[threadIdx.x] = d.y;
  }
  __syncthreads();
  const int q = heads[p];
  if (q < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 1;                                         // parts: this pair's and those of the pairs after it
  for (uint32_t more = 1; more;) {
    const int i = p + n + lane;
    const uint32_t other = __ballot_sync(0xffffffffu, i >= pairs || tails[i] != q);
    n += other ? __ffs(other) - 1 : 32;
    more = other == 0;
  }
  const int h = blockIdx.y * 32 + lane;
  constexpr int UL = 8, U = 4;
  auto part = [&](int i) { return static_cast<size_t>(2 * (p + i) + (i == 0)); };
  float m = -INFINITY;
  for (int i = 0; i < n; i += UL) {
    float l[UL];
#pragma unroll
    for (int k = 0; k < UL; ++k) l[k] = i + k < n ? l_part[part(i + k) * H + h] : -INFINITY;
#pragma unroll
    for (int k = 0; k < UL; ++k) m = fmaxf(m, l[k]);
  }
  const float m_eff = m == -INFINITY ? 0.f : m;
  float tot = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int d4 = blockIdx.z * 32 + 4 * warp + 2 * t;
    float acc[8] = {};
    tot = 0.f;
    for (int i = 0; i < n; i += U) {
      float l[U];
      float4 a[U], b[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const bool is = i + k < n;
        const float4* src = reinterpret_cast<const float4*>(o_part) + (part(i + k) * (DSA_DIM_V / 4) + d4) * H + h;
        l[k] = is ? l_part[part(i + k) * H + h] : -INFINITY;
        a[k] = is ? src[0] : make_float4(0.f, 0.f, 0.f, 0.f);
        b[k] = is ? src[H] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float w = expf(l[k] - m_eff);
        tot += w;
        acc[0] = fmaf(w, a[k].x, acc[0]);
        acc[1] = fmaf(w, a[k].y, acc[1]);
        acc[2] = fmaf(w, a[k].z, acc[2]);
        acc[3] = fmaf(w, a[k].w, acc[3]);
        acc[4] = fmaf(w, b[k].x, acc[4]);
        acc[5] = fmaf(w, b[k].y, acc[5]);
        acc[6] = fmaf(w, b[k].z, acc[6]);
        acc[7] = fmaf(w, b[k].w, acc[7]);
      }
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    turn[lane][2 * warp + t] =
        make_uint4(bf16x2_bits(acc[0] * inv, acc[1] * inv), bf16x2_bits(acc[2] * inv, acc[3] * inv),
                   bf16x2_bits(acc[4] * inv, acc[5] * inv), bf16x2_bits(acc[6] * inv, acc[7] * inv));
  }
  if (blockIdx.z == 0 && warp == 0) lse[static_cast<size_t>(q) * H + h] = tot == 0.f ? -INFINITY : m_eff + logf(tot);
  __syncthreads();
  const int r = threadIdx.x >> 3, c = threadIdx.x & 7;
  uint4* dst = reinterpret_cast<uint4*>(out + (static_cast<size_t>(q) * H + blockIdx.y * 32 + r) * DSA_DIM_V + 128 * blockIdx.z);
  dst[c] = turn[r][c];
  dst[c + 8] = turn[r][c + 8];
}

constexpr size_t DESC_OFF = 256;
constexpr size_t L_OFF = DESC_OFF + 2 * MAX_PAIRS * 4 + 176;      // 1024
static_assert(L_OFF % 256 == 0, "aligned");

template <bool KV8, bool IDX>
cudaError_t launch(const AttendArgs& a, const AttendMaps& m, int pairs, cudaStream_t st) {
  static std::atomic<bool> done[64];
  auto kernel = attend_kernel<KV8, IDX>;
  const cudaError_t e = set_once_per_device(done, [kernel] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<KV8>::SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(Plan<KV8>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Plan<KV8>::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  unsigned int na = 1;
  add_pdl_attr(attr, &na, true);                     // its barriers and tensor memory beside the end of the kernel before
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, kernel, a, m);
}

}  // namespace

size_t attend_workspace_bytes(int H) {
  const size_t parts = 2 * MAX_PAIRS;
  return L_OFF + parts * H * 4 + parts * H * DSA_DIM_V * 4;
}

cudaError_t launch_attend(const __nv_bfloat16* q, const void* pool, const float* kv_scales, int num_pages,
                          int page_size, int scale_block, const int32_t* page_table, int max_pages,
                          const int32_t* q_offsets, const int32_t* q_vis, const int32_t* idx, int topk, int B,
                          int Q, int H, int sinks, int window, float scale, __nv_bfloat16* out, float* lse,
                          void* ws, cudaStream_t st) {
  AttendArgs a = {};
  a.q = q;
  a.pool = static_cast<const uint8_t*>(pool);
  a.kv_scales = kv_scales;
  a.page_table = page_table;
  a.q_offsets = q_offsets;
  a.q_vis = q_vis;
  a.idx = idx;
  a.out = out;
  a.lse = lse;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.err = reinterpret_cast<uint32_t*>(w);
  a.desc = reinterpret_cast<int32_t*>(w + DESC_OFF);
  a.l_part = reinterpret_cast<float*>(w + L_OFF);
  a.o_part = a.l_part + 2 * MAX_PAIRS * H;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  while (kv_scales && (1 << a.block_shift) < scale_block) ++a.block_shift;
  a.B = B;
  a.Q = Q;
  a.H = H;
  a.topk = topk;
  a.sinks = sinks;
  a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  const int sms = device_sm_count() / 2;
  const int pairs = sms < 1 ? 1 : (sms < MAX_PAIRS ? sms : MAX_PAIRS);
  AttendMaps m = {};
  const uint64_t pool_rows = static_cast<uint64_t>(num_pages) * page_size;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  bool ok = encode_tiled_2d(&m.q, bf, q, DSA_DIM, static_cast<uint64_t>(Q) * H, DSA_DIM * 2, 64, H / 2);
  // boxes of several rows are used where the rows are consecutive
  if (kv_scales) {
    const CUtensorMapSwizzle flat = CU_TENSOR_MAP_SWIZZLE_NONE;
    const CUtensorMapDataType u32 = CU_TENSOR_MAP_DATA_TYPE_UINT32;
    ok = ok && encode_tiled_2d(&m.row, u8, pool, DSA_DIM, pool_rows, DSA_DIM, 256, 1, flat) &&
         encode_tiled_2d(&m.run, u8, pool, DSA_DIM, pool_rows, DSA_DIM, 256, RUN, flat) &&
         encode_tiled_2d(&m.row_hi, u32, pool, DSA_DIM / 4, pool_rows, DSA_DIM, 80, 1, flat) &&
         encode_tiled_2d(&m.run_hi, u32, pool, DSA_DIM / 4, pool_rows, DSA_DIM, 80, RUN, flat);
  } else {
    ok = ok && encode_tiled_2d(&m.row, bf, pool, DSA_DIM, pool_rows, DSA_DIM * 2, 64, 1) &&
         encode_chunks_bf16(&m.run, pool, KC, pool_rows, DSA_DIM * 2, 8, 3) &&
         encode_chunks_bf16(&m.run_hi, pool, KC, pool_rows, DSA_DIM * 2, RUN, 4);
  }
  if (!ok) return cudaErrorInvalidValue;
  cudaError_t e = idx ? launch<true, true>(a, m, pairs, st)
                      : (kv_scales ? launch<true, false>(a, m, pairs, st) : launch<false, false>(a, m, pairs, st));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(H / 32), DSA_DIM_V / 128);
  cfg.blockDim = dim3(MT, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  unsigned int na = 0;
  add_pdl_attr(attr, &na, true);
  cfg.attrs = attr;
  cfg.numAttrs = na;
  return cudaLaunchKernelEx(&cfg, attend_merge_kernel, static_cast<const int32_t*>(a.desc),
                            static_cast<const float*>(a.o_part), static_cast<const float*>(a.l_part), H, out, lse);
}

}  // namespace dsa
