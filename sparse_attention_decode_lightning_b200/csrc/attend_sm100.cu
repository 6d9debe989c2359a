// MLA decode attention over a list of cached tokens, on sm_100a tensor cores:
// the window-and-sinks and the block-scaled selected forms.  Per head h of
// query q, over the tokens j of its list:
//   z_j = scale * q[h, 0:576] . C[j, 0:576],  O[h] = sum_j softmax(z)_j C[j, 0:512],
//   LSE[h] = ln sum_j exp(z_j);   an empty list gives O = 0, LSE = -inf.
// The list is the first `sinks` and the last `window` visible positions
// (RANGE), or a row of selected positions (IDX).  The cache is bf16, or e4m3
// codes with an fp32 scale s_j for each block of tokens: C[j] = s_j * code[j].
//
// One pass over the list in tiles of 64 tokens.  A CTA owns 256 of the 512
// value dims and every query head (M = 128; 64 heads leave the upper rows
// zero), so the scores of a tile are computed by the two CTAs of a pair, and
// nothing crosses between them: 36 score steps and 16 value steps of 32 and
// 128 tensor cycles a tile, 1664, where an undivided tile would need 1088 a
// CTA.  What it saves is an exchange of scores in the middle of each tile's
// chain, which set the pace of the gathered kernel of sparse_mla_sm100.cu.
//
// The work is cut evenly: the tiles of all queries, one after another, are
// divided over the SM pairs, so ragged lists leave no pair idle; a query whose
// tiles lie on several pairs leaves partial results that a second kernel
// merges by log-sum-exp.
//
// Operands.  bf16 cache: q, C and P as bf16 (P's rounding, 2^-9 of each
// weight, is the size of the output's own).  e4m3 cache: codes widened to fp16
// (exact), q scaled by a power of two a head so that its largest element lies
// in [2^14, 2^15) and rounded to fp16 (exact for all that is not 2^-28 times
// smaller), P as fp16.  The scales enter in fp32: z_j takes s_j, and P_j is
// formed as exp2(z_j + log2 s_j - m) with m the running maximum of that sum,
// so that P <= 2^8 whatever the scales are; l sums P_j / s_j.  Sums, maxima
// and O are fp32.
//
// Tensor memory (512 columns): O [0,256) | scores slot 0 [256,320) | slot 1
// [320,384) | the 256 query dims that are also this CTA's value dims [384,512).
// P overwrites its slot's scores.  Shared memory: the other 320 query dims
// (80 KB), three stages of value chunks (4 x 8 KB each), one stage of the 5
// other chunks of a tile, refilled by halves while the tile's values run.  A
// chunk is 64 tokens x 64 dims, 16 bits, in the 128-byte swizzle.
//
// Roles (512 threads): warp 0 issues the MMAs; warps 1..3 look up the pool
// rows (list -> page table -> scale) up to six tiles ahead, since each is a
// chain of dependent loads; warps 4..7 softmax, rescale and output, one head a
// thread; warps 8..15 load queries and tiles.  Rows that the list does not
// hold are filled with zeros and never read, so that what lies in the cache
// there (NaN, say) cannot reach a product.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace dsa {
namespace {

constexpr int NR = 64;                               // tokens per tile
constexpr int CH = NR * 128;                         // chunk bytes: 64 tokens x 64 dims x 2
constexpr int QCH = 128 * 128;                       // query chunk bytes: 128 heads x 64 dims x 2
constexpr int AC = 4;                                // latent chunks of a tile that are scores only
constexpr int VC = 4;                                // chunks that are values too (one more: positions)
constexpr int NV = 3;                                // value stages
constexpr int RR = 6;                                // tiles looked up ahead
constexpr int RESOLVERS = 3;
constexpr int SMX = 4;                               // softmax warps
constexpr int GROUP = 4;                             // warps of each of the two loader groups
constexpr int LOADERS = 2 * GROUP;
constexpr int THREADS = 32 * (1 + RESOLVERS + SMX + LOADERS);

constexpr int OFF_QX = 0;
constexpr int OFF_V = OFF_QX + (AC + 1) * QCH;       // [3][4] value chunks
constexpr int OFF_A = OFF_V + NV * VC * CH;          // [5] chunks of the other half, and the positions
constexpr int OFF_COL = OFF_A + (AC + 1) * CH;       // float4 [RR][64]: scale, log2 s, 1 / s of each token
constexpr int OFF_TILE = OFF_COL + RR * NR * 16;     // float4 [RR]: the same for a whole tile; w: it holds
constexpr int OFF_ROWS = OFF_TILE + RR * 16;         // int32 [RR][64]: pool row or -1
constexpr int OFF_FOLD = OFF_ROWS + RR * NR * 4;     // uint16 [RR][64]: fp16 factor of a token's codes
constexpr int OFF_MASK = OFF_FOLD + RR * NR * 2;     // uint32 [RR][2]: tokens that count
constexpr int OFF_QMUL = OFF_MASK + RR * 2 * 4;      // float [128]
constexpr int OFF_SCAN = OFF_QMUL + 128 * 4;         // int64 [17], then the first query and its tile
constexpr int OFF_BAR = OFF_SCAN + 20 * 8;
constexpr int NBAR = 2 * RR + 4 * 2 + 2 * NV + 3;
constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory exceeds the sm_100 limit");
static_assert(4 * QCH <= NV * VC * CH, "the query's value-dim chunks pass through the value stages");
static_assert(OFF_V % 1024 == 0 && OFF_A % 1024 == 0, "swizzle atoms");
constexpr uint32_t O_COL = 0, S_COL = 256, Q_COL = 384, TMEM_COLS = 512;

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

// first the sinks, then the window of query with `vis` visible tokens
struct List {
  int n;            // tokens
  int ns;           // of them sinks: entry j < ns is position j
  int w0;           // entry j >= ns is position w0 + j - ns
};

__device__ __forceinline__ int visible(const AttendArgs& a, int q) {
  const int v = max(0, __ldg(a.q_vis + q));
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_shift;
  return v < cap ? v : static_cast<int>(cap);
}

__device__ __forceinline__ List list_of(const AttendArgs& a, int vis) {
  List l;
  l.ns = min(a.sinks, vis);
  l.w0 = max(l.ns, vis - a.window);
  l.n = l.ns + vis - l.w0;
  return l;
}

// tiles of query q: at least one, which writes the result of an empty list
template <bool IDX>
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int q) {
  if constexpr (IDX) return (a.topk + NR - 1) / NR;
  return max(1, (list_of(a, visible(a, q)).n + NR - 1) / NR);
}

__device__ __forceinline__ int seq_of_query(const int32_t* q_offsets, int B, int q, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const uint32_t m = __ballot_sync(0xffffffffu, i < hi && __ldg(q_offsets + i) <= q);
    if (m == 0) break;                     // q lies before the first sequence
    lo += (31 - __clz(m)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

__device__ __forceinline__ bool wwait(uint64_t* bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err));
}

__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// four e4m3 codes -> four fp16 times f (a power of two), exactly
__device__ __forceinline__ uint2 widen4(uint32_t w, __half2 f) {
  const __half2 a = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3)), f);
  const __half2 b = __hmul2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)), f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
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

// larger magnitude bits of a bf16 pair's two values, seen as two u16
__device__ __forceinline__ uint32_t mag2(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

__device__ __forceinline__ uint32_t scale_pair(uint32_t w, float s) {
  return f16x2_bits(__uint_as_float(w << 16) * s, __uint_as_float(w & 0xFFFF0000u) * s);
}

template <bool KV8, bool IDX>
__global__ void __launch_bounds__(THREADS, 1) attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* qx = smem + OFF_QX;
  uint8_t* vst = smem + OFF_V;
  uint8_t* ast = smem + OFF_A;
  int* rows = reinterpret_cast<int*>(smem + OFF_ROWS);
  float4* col = reinterpret_cast<float4*>(smem + OFF_COL);
  float4* tsc = reinterpret_cast<float4*>(smem + OFF_TILE);
  uint16_t* fold = reinterpret_cast<uint16_t*>(smem + OFF_FOLD);
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + OFF_MASK);
  float* qmul = reinterpret_cast<float*>(smem + OFF_QMUL);
  int64_t* scan = reinterpret_cast<int64_t*>(smem + OFF_SCAN);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* r_full = bars;                 // [RR] rows of a tile are looked up
  uint64_t* r_empty = r_full + RR;
  uint64_t* a_full = r_empty + RR;         // [2] chunks 0, 1 of a tile, then 2, 3 and the positions
  uint64_t* a_empty = a_full + 2;          // [2] the scores have read them
  uint64_t* s_full = a_empty + 2;          // [2] scores of a tile are in their slot
  uint64_t* p_full = s_full + 2;           // [2] P of a tile is in its slot
  uint64_t* v_full = p_full + 2;           // [NV] a tile's value chunks
  uint64_t* v_free = v_full + NV;          // [NV] the value MMA is done: its stage and scores slot are free
  uint64_t* q_staged = v_free + NV;        // a segment's query is in shared memory
  uint64_t* q_ready = q_staged + 1;        // ... and its value dims in tensor memory
  uint64_t* o_final = q_ready + 1;         // every MMA of a segment is done
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + OFF_MISC);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  pdl_trigger();

  if (tid == 0) {
    for (int i = 0; i < RR; ++i) {
      mbar_init(&r_full[i], 1);
      mbar_init(&r_empty[i], LOADERS + SMX);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_full[i], GROUP);
      mbar_init(&a_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], SMX);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(&v_full[i], GROUP);
      mbar_init(&v_free[i], 1);
    }
    mbar_init(q_staged, LOADERS);
    mbar_init(q_ready, SMX);
    mbar_init(o_final, 1);
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(tmem_holder, TMEM_COLS);

  // This pair's share [t0, t1) of all tiles: a thread sums the tiles of some
  // consecutive queries, the block scans the sums.
  const int per = (a.Q + THREADS - 1) / THREADS;
  const int qa = min(a.Q, tid * per), qb = min(a.Q, qa + per);
  int64_t sum = 0;
  for (int q = qa; q < qb; ++q) sum += tiles_of<IDX>(a, q);
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int64_t base = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) base = total;
    total += scan[w];
  }
  base += incl - sum;
  const int64_t np = total < pairs ? total : pairs;       // pairs that get work
  const int64_t t0 = pair < np ? total * pair / np : 0;
  const int64_t t1 = pair < np ? total * (pair + 1) / np : 0;
  if (t1 > t0 && t0 >= base && t0 < base + sum) {
    int64_t at = base;
    int q = qa;
    for (int n; at + (n = tiles_of<IDX>(a, q)) <= t0; ++q) at += n;
    scan[17] = q;
    scan[18] = t0 - at;
  }
  if (half == 0 && tid < 2 && t1 == t0) a.desc[2 * pair + tid] = -1;
  __syncthreads();
  const uint32_t tmem = *tmem_holder;
  const int q0 = static_cast<int>(scan[17]);
  const int off0 = static_cast<int>(scan[18]);
  const int ntile = static_cast<int>(t1 - t0);

  if (warp == 0) {
    // ------------------------------------------------------------ MMA issuer
    // The warp walks together, so that descriptors stay in uniform registers,
    // and one elected lane issues.  The loaders fence their own writes.
    constexpr uint32_t fmt = KV8 ? 0u /*F16*/ : 1u /*BF16*/;
    constexpr uint32_t idesc_s = umma_idesc(fmt, 128, NR);
    constexpr uint32_t idesc_pv = umma_idesc(fmt, 128, 256, 0, 1);
    const uint64_t dq = umma_desc_sw128(smem_u32(qx), 1024, 16);
    const uint64_t da = umma_desc_sw128(smem_u32(ast), 1024, 16);
    const uint64_t dv = umma_desc_sw128(smem_u32(vst), 1024, 16);
    const uint64_t dm = umma_desc_sw128_mn(smem_u32(vst), CH, 1024);
    const bool lead = elect_one();
    bool ok = true;
    int q = q0, off = off0, left = ntile;
    uint32_t g = 0;                              // tiles so far
    for (uint32_t seg = 0; left > 0 && ok; ++seg, ++q, off = 0) {
      const int n = min(tiles_of<IDX>(a, q) - off, left);
      left -= n;
      if (!(ok = wwait(q_ready, seg & 1, a.err))) break;
      tc_fence_after();
      // values of tile u - 1 between the scores of tile u, so that neither the
      // softmax before nor the free slot after is waited for
      for (int u = 0; u <= n && ok; ++u) {
        const uint32_t gu = g + u, sb = gu & 1, vs = gu % NV;
        const uint32_t d = tmem + S_COL + sb * NR;
        if (u < n) {
          // P of tile u - 2 has left the slot
          if (gu >= 2 && !(ok = wwait(&v_free[(gu - 2) % NV], ((gu - 2) / NV) & 1, a.err))) break;
          if (!(ok = wwait(&a_full[0], gu & 1, a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16(d, dq + (k >> 2) * (QCH >> 4) + (k & 3) * 2, da + (k >> 2) * (CH >> 4) + (k & 3) * 2, idesc_s,
                      k > 0);
            mma_commit(&a_empty[0]);
          }
          __syncwarp();
          if (!(ok = wwait(&a_full[1], gu & 1, a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 8; k < 4 * (AC + 1); ++k)
              mma_f16(d, dq + (k >> 2) * (QCH >> 4) + (k & 3) * 2, da + (k >> 2) * (CH >> 4) + (k & 3) * 2, idesc_s,
                      1u);
            mma_commit(&a_empty[1]);
          }
          __syncwarp();
          if (!(ok = wwait(&v_full[vs], (gu / NV) & 1, a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_f16_ts(d, tmem + Q_COL + k * 8, dv + vs * (VC * CH >> 4) + (k >> 2) * (CH >> 4) + (k & 3) * 2,
                         idesc_s, 1u);
          }
          __syncwarp();
        }
        if (u >= 1) {
          const uint32_t gt = gu - 1, tb = gt & 1, ts = gt % NV;
          if (!(ok = wwait(&p_full[tb], (gt >> 1) & 1, a.err))) break;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int k = 0; k < NR / 16; ++k)
              mma_f16_ts(tmem + O_COL, tmem + S_COL + tb * NR + k * 8, dm + ts * (VC * CH >> 4) + k * (2048 >> 4),
                         idesc_pv, (u > 1 || k > 0) ? 1u : 0u);
            mma_commit(&v_free[ts]);
            if (u == n) mma_commit(o_final);
          }
          __syncwarp();
        }
        if (u < n) {
          if (lead) {
#pragma unroll
            for (int k = 8; k < 4 * VC; ++k)
              mma_f16_ts(d, tmem + Q_COL + k * 8, dv + vs * (VC * CH >> 4) + (k >> 2) * (CH >> 4) + (k & 3) * 2,
                         idesc_s, 1u);
            mma_commit(&s_full[sb]);
          }
          __syncwarp();
        }
      }
      g += n;
    }
  } else if (warp < 1 + RESOLVERS) {
    // ------------------------------------------------------------ row look-up
    bool ok = true;
    int q = q0, off = off0, left = ntile;
    uint32_t g = 0;
    while (left > 0 && ok) {
      const int n = min(tiles_of<IDX>(a, q) - off, left);
      left -= n;
      const int b = seq_of_query(a.q_offsets, a.B, q, lane);
      const int vis = visible(a, q);
      if (__ldg(a.q_vis + q) > vis && lane == 0) raise_error(a.err, DEVERR_BOUNDS);
      const List ls = list_of(a, vis);
      for (int u = 0; u < n; ++u, ++g) {
        if (g % RESOLVERS != static_cast<uint32_t>(warp - 1)) continue;
        const uint32_t slot = g % RR;
        int row[2];
        float s[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = (off + u) * NR + 32 * i + lane;
          int pos = -1;
          if constexpr (IDX) {
            if (j < a.topk) pos = __ldg(a.idx + static_cast<size_t>(q) * a.topk + j);
          } else {
            if (j < ls.n) pos = j < ls.ns ? j : ls.w0 + (j - ls.ns);
          }
          row[i] = -1;
          s[i] = 1.f;
          if (pos >= 0 && pos < vis) {
            const int pg = __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + (pos >> a.page_shift));
            if (pg >= 0 && pg < a.num_pages) {
              row[i] = (pg << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
              if constexpr (KV8) {
                s[i] = __ldg(a.kv_scales + (row[i] >> a.block_shift));
                if (!(s[i] >= 0x1p-40f && s[i] <= 0x1p40f)) row[i] = -1;
              }
            }
          }
          if (row[i] < 0 && pos != -1) raise_error(a.err, DEVERR_BOUNDS);
        }
        ok = wwait(&r_empty[slot], ((g / RR) & 1) ^ 1, a.err);
        if (!ok) break;
        if constexpr (KV8) {
          // Scales that differ by powers of two, up to 2^15, go into the fp16
          // codes, exactly (a code is a multiple of 2^-9, fp16's least step is
          // 2^-24): the tile then has one scale, its largest.  Other tiles keep
          // one a token.
          uint32_t lo = 0xffffffffu, hi = 0, mlo = 0xffffffffu, mhi = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t bits = __float_as_uint(s[i]);
            if (row[i] >= 0) {
              lo = min(lo, bits);
              hi = max(hi, bits);
              mlo = min(mlo, bits & 0x7FFFFFu);
              mhi = max(mhi, bits & 0x7FFFFFu);
            }
          }
          lo = __reduce_min_sync(0xffffffffu, lo);
          hi = __reduce_max_sync(0xffffffffu, hi);
          mlo = __reduce_min_sync(0xffffffffu, mlo);
          mhi = __reduce_max_sync(0xffffffffu, mhi);
          const bool one = hi == 0 || (mlo == mhi && (hi - lo) >> 23 <= 15);
          const float st = hi == 0 ? 1.f : __uint_as_float(hi);
          if (lane == 0)
            tsc[slot] = make_float4(st * a.scale_log2, log2f(st), __fdiv_rn(1.f, st), one ? 1.f : 0.f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t down = one && row[i] >= 0 ? (hi - __float_as_uint(s[i])) >> 23 : 0u;
            fold[slot * NR + 32 * i + lane] = down < 15 ? static_cast<uint16_t>((15 - down) << 10) : uint16_t{0x200};
            if (!one)
              col[slot * NR + 32 * i + lane] =
                  row[i] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                             : make_float4(s[i] * a.scale_log2, log2f(s[i]), __fdiv_rn(1.f, s[i]), 0.f);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rows[slot * NR + 32 * i + lane] = row[i];
          const uint32_t m = __ballot_sync(0xffffffffu, row[i] >= 0);
          if (lane == 0) mask[slot * 2 + i] = m;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&r_full[slot]);
      }
      ++q;
      off = 0;
    }
  } else if (warp < 1 + RESOLVERS + SMX) {
    // ------------------------------------------------------------ softmax, output
    const int quarter = warp & 3;
    const int h = quarter * 32 + lane;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    bool ok = true;
    int q = q0, off = off0, left = ntile;
    uint32_t g = 0;
    int head_q = -1, tail_q = -1;                    // queries this pair holds a part of
    for (uint32_t seg = 0; left > 0 && ok; ++seg, ++q, off = 0) {
      const int nt = tiles_of<IDX>(a, q);
      const int n = min(nt - off, left);
      left -= n;
      // the query's value dims, staged by the loaders, go to tensor memory
      ok = wwait(q_staged, seg & 1, a.err);
      for (int c = 0; c < VC; ++c) {
        float w[32];
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint4 v = *reinterpret_cast<const uint4*>(vst + c * QCH + h * 128 + ((p ^ (h & 7)) << 4));
          w[4 * p] = __uint_as_float(v.x);
          w[4 * p + 1] = __uint_as_float(v.y);
          w[4 * p + 2] = __uint_as_float(v.z);
          w[4 * p + 3] = __uint_as_float(v.w);
        }
        tmem_st32(lane_base + Q_COL + c * 32, w);
      }
      const float qm = KV8 ? qmul[h] : 1.f;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);

      float m_use = -INFINITY, l = 0.f;
      for (int u = 0; u < n; ++u, ++g) {
        const uint32_t sb = g & 1, slot = g % RR;
        if (ok) ok = wwait(&r_full[slot], (g / RR) & 1, a.err);
        if (ok) ok = wwait(&s_full[sb], (g >> 1) & 1, a.err);
        tc_fence_after();
        float z[NR];
        tmem_ld32(lane_base + S_COL + sb * NR, z);
        tmem_ld32(lane_base + S_COL + sb * NR + 32, z + 32);
        tmem_ld_wait();
        const uint32_t m0 = mask[slot * 2], m1 = mask[slot * 2 + 1];
        const float4* cp = col + slot * NR;
        float4 ts = make_float4(a.scale_log2, 0.f, 1.f, 1.f);
        if constexpr (KV8) ts = tsc[slot];
        if (!KV8 || ts.w != 0.f) {
          const float k = ts.x * qm;
#pragma unroll
          for (int j = 0; j < NR; ++j) z[j] = fmaf(z[j], k, ts.y);
        } else {
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            const float2 k = *reinterpret_cast<const float2*>(cp + j);
            z[j] = fmaf(z[j] * qm, k.x, k.y);
          }
        }
        if ((m0 & m1) != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            z[j] = ((m0 >> j) & 1u) ? z[j] : -INFINITY;
            z[32 + j] = ((m1 >> j) & 1u) ? z[32 + j] : -INFINITY;
          }
        }
        float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < NR; ++j) mt[j & 3] = fmaxf(mt[j & 3], z[j]);
        const float mtile = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
        // the maximum that P refers to moves only when it falls 8 behind (a
        // factor of 2^8, which fp16 holds), so O is seldom rescaled
        float alpha = 1.f;
        bool resc = false;
        if (mtile > m_use + 8.f) {
          if (m_use != -INFINITY) {
            alpha = fast_exp2(m_use - mtile);
            resc = true;
          }
          m_use = mtile;
        }
        const float m_eff = m_use == -INFINITY ? 0.f : m_use;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float* zh = z + 32 * hh;
#pragma unroll
          for (int j = 0; j < 32; ++j) zh[j] = fast_exp2(zh[j] - m_eff);
          if (!KV8 || ts.w != 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) ps[j & 3] += zh[j];
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) ps[j & 3] = fmaf(zh[j], cp[32 * hh + j].z, ps[j & 3]);
          }
          float pk[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[j] = __uint_as_float(KV8 ? f16x2_bits(zh[2 * j], zh[2 * j + 1]) : bf16x2_bits(zh[2 * j], zh[2 * j + 1]));
          tmem_st16(lane_base + S_COL + sb * NR + 16 * hh, pk);
        }
        l = fmaf(l, alpha, ((ps[0] + ps[1]) + (ps[2] + ps[3])) * (KV8 && ts.w != 0.f ? ts.z : 1.f));
        __syncwarp();
        if (lane == 0) mbar_arrive(&r_empty[slot]);
        if (__any_sync(0xffffffffu, resc)) {
          // after the value MMA of the tile before
          if (ok) ok = wwait(&v_free[(g - 1) % NV], ((g - 1) / NV) & 1, a.err);
          tc_fence_after();
          for (int c = 0; c < 8; ++c) {
            float o[32];
            tmem_ld32(lane_base + O_COL + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tmem_st32(lane_base + O_COL + c * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
      }
      // ---- the segment's result: the query's own, or a part of it
      if (ok) ok = wwait(o_final, seg & 1, a.err);
      tc_fence_after();
      const bool whole = n == nt;
      const bool head = off == 0;
      const int part = 2 * pair + (head ? 1 : 0);
      if (!whole) (head ? head_q : tail_q) = q;
      const bool live = h < a.H;
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;   // NaN stays NaN
      const bool none = l == 0.f;
      for (int c = 0; c < 8; ++c) {
        float o[32];
        tmem_ld32(lane_base + O_COL + c * 32, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i] * inv;
        if (!live) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + (static_cast<size_t>(q) * a.H + h) * DSA_DIM_V + 256 * half + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(bf16x2_bits(o[8 * i], o[8 * i + 1]), bf16x2_bits(o[8 * i + 2], o[8 * i + 3]),
                                bf16x2_bits(o[8 * i + 4], o[8 * i + 5]), bf16x2_bits(o[8 * i + 6], o[8 * i + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(a.o_part + (static_cast<size_t>(part) * a.H + h) * DSA_DIM_V + 256 * half + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (half == 0 && live)
        (whole ? a.lse + static_cast<size_t>(q) * a.H + h : a.l_part + static_cast<size_t>(part) * a.H + h)[0] =
            none ? -INFINITY : (m_use + log2f(l)) * 0.69314718055994531f;
      tc_fence_before();                             // O was read before the next segment writes it
    }
    if (half == 0 && quarter == 0 && lane == 0 && ntile > 0) {
      a.desc[2 * pair] = tail_q;
      a.desc[2 * pair + 1] = head_q;
    }
  } else {
    // ------------------------------------------------------------ loaders
    // Two groups of four warps, so that neither waits for the other's stage:
    // group 0 fills the scores-only chunks (one stage, handed over in halves),
    // group 1 the value chunks (three stages).
    const int lw = warp - (1 + RESOLVERS + SMX);
    const bool vals = lw >= GROUP;
    const int lt = (lw & (GROUP - 1)) * 32 + lane;
    bool ok = true;
    int q = q0, off = off0, left = ntile;
    uint32_t g = 0;
    for (uint32_t seg = 0; left > 0 && ok; ++seg, ++q, off = 0) {
      const int n = min(tiles_of<IDX>(a, q) - off, left);
      left -= n;
      if (seg > 0) ok = wwait(o_final, (seg - 1) & 1, a.err);
      if (!ok) break;
      // the query: a warp takes 16 heads, four at a time; 72 pieces of 8 dims
      // a head.  Chunks of this CTA's value dims pass through the value stages.
      for (int h0 = 16 * lw; h0 < 16 * lw + 16; h0 += 4) {
        uint4 v[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4* src = reinterpret_cast<const uint4*>(a.q + (static_cast<size_t>(q) * a.H + h0 + i) * DSA_DIM);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            v[i][k] = h0 + i < a.H && (k < 2 || lane < 8) ? __ldg(src + 32 * k + lane) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = h0 + i;
          if constexpr (KV8) {
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 3; ++k) m = mag2(mag2(mag2(mag2(m, v[i][k].x), v[i][k].y), v[i][k].z), v[i][k].w);
            m = max(m & 0xFFFFu, m >> 16);
            m = __reduce_max_sync(0xffffffffu, m);
            // largest element in [2^14, 2^15); infinities and NaN stay what they are
            const int e = min(max(static_cast<int>(m >> 7), 14), 254);
            const float s = m == 0 || m >= 0x7F80u ? 1.f : __uint_as_float(static_cast<uint32_t>(min(254, 268 - e)) << 23);
#pragma unroll
            for (int k = 0; k < 3; ++k)
              v[i][k] = make_uint4(scale_pair(v[i][k].x, s), scale_pair(v[i][k].y, s), scale_pair(v[i][k].z, s),
                                   scale_pair(v[i][k].w, s));
            if (lane == 0) qmul[h] = __fdiv_rn(1.f, s);
          }
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            if (k == 2 && lane >= 8) continue;
            const int p = 32 * k + lane, c = p >> 3;
            const int sw = h * 128 + (((p & 7) ^ (h & 7)) << 4);
            const int x = c == 8 ? AC : (c & 3);
            uint8_t* dst = c < 8 && (c >> 2) == half ? vst + (c & 3) * QCH : qx + x * QCH;
            *reinterpret_cast<uint4*>(dst + sw) = v[i][k];
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_staged);

      auto wait_a = [&](uint32_t gg, int part) { return wwait(&a_empty[part], (gg & 1) ^ 1, a.err); };
      auto wait_v = [&](uint32_t gg, bool first) {
        if (first && !wwait(q_ready, seg & 1, a.err)) return false;   // the query has left the stages
        return wwait(&v_free[gg % NV], ((gg / NV) & 1) ^ 1, a.err);
      };
      auto done = [&](uint64_t* bar) {                               // the writes are for the tensor core
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      if constexpr (KV8) {
        // thread: 16 + 16 codes of each chunk of one token; a tile's pieces are
        // all in flight before the tile before is widened and stored.  The
        // rows of a quarter warp, r & 7 in {0,1,4,5} or {2,3,6,7}, put its 16-byte
        // stores into eight different bank groups.
        const int rj = lt >> 1, u2 = lt & 1;
        const int r = (rj & ~7) | (rj & 1) | ((rj & 2) << 1) | ((rj & 4) >> 1);
        uint4 va[2 * (AC + 1)], vb[2 * (AC + 1)];
        __half2 fa, fb;
        auto fetch = [&](uint4* v, __half2& f, uint32_t gg) {
          const uint32_t slot = gg % RR;
          ok = ok && wwait(&r_full[slot], (gg / RR) & 1, a.err);
          const int row = ok ? rows[slot * NR + r] : -1;
          f = __half2half2(__ushort_as_half(fold[slot * NR + r]));
          const uint4* src = reinterpret_cast<const uint4*>(a.pool + static_cast<size_t>(row < 0 ? 0 : row) * DSA_DIM) + u2;
          const int c0 = 4 * (vals ? half : half ^ 1);
#pragma unroll
          for (int c = 0; c < AC + 1; ++c) {
            const int dc = c < 4 ? c0 + c : 8;
            const bool get = row >= 0 && (c < 4 || !vals);
            v[2 * c] = get ? __ldg(src + 4 * dc) : make_uint4(0u, 0u, 0u, 0u);
            v[2 * c + 1] = get ? __ldg(src + 4 * dc + 2) : make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&r_empty[slot]);
        };
        // pieces 2 u2 + {0, 1} and 4 + 2 u2 + {0, 1} of token r's 128 bytes
        auto put = [&](uint8_t* dst, const uint4* v, __half2 f) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint2 a0 = widen4(v[i].x, f), a1 = widen4(v[i].y, f), a2 = widen4(v[i].z, f), a3 = widen4(v[i].w, f);
            const int p = 4 * i + 2 * u2;
            *reinterpret_cast<uint4*>(dst + r * 128 + ((p ^ (r & 7)) << 4)) = make_uint4(a0.x, a0.y, a1.x, a1.y);
            *reinterpret_cast<uint4*>(dst + r * 128 + (((p + 1) ^ (r & 7)) << 4)) = make_uint4(a2.x, a2.y, a3.x, a3.y);
          }
        };
        auto store = [&](const uint4* v, __half2 f, uint32_t gg, bool first) {
          if (vals) {
            if (!(ok = wait_v(gg, first))) return;
#pragma unroll
            for (int c = 0; c < VC; ++c) put(vst + (gg % NV) * (VC * CH) + c * CH, v + 2 * c, f);
            done(&v_full[gg % NV]);
          } else {
            if (!(ok = wait_a(gg, 0))) return;
#pragma unroll
            for (int c = 0; c < 2; ++c) put(ast + c * CH, v + 2 * c, f);
            done(&a_full[0]);
            if (!(ok = wait_a(gg, 1))) return;
#pragma unroll
            for (int c = 2; c < AC + 1; ++c) put(ast + c * CH, v + 2 * c, f);
            done(&a_full[1]);
          }
        };
        fetch(va, fa, g);
        for (int u = 0; u < n && ok; u += 2) {
          if (u + 1 < n) fetch(vb, fb, g + u + 1);
          if (ok) store(va, fa, g + u, u == 0);
          if (u + 1 < n && ok) {
            if (u + 2 < n) fetch(va, fa, g + u + 2);
            if (ok) store(vb, fb, g + u + 1, false);
          }
        }
      } else {
        // thread: 16 bytes of each chunk of four tokens, copied without registers
        const int p = lt & 7, r0 = lt >> 3;
        for (int u = 0; u < n && ok; ++u) {
          const uint32_t gg = g + u, slot = gg % RR;
          ok = wwait(&r_full[slot], (gg / RR) & 1, a.err);
          if (!ok) break;
          int row[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) row[i] = rows[slot * NR + r0 + 16 * i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&r_empty[slot]);
          auto copy = [&](uint8_t* dst, int dc) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = r0 + 16 * i;                             // r & 7 == r0 & 7
              cp_async16(dst + r * 128 + ((p ^ (r0 & 7)) << 4),
                         a.pool + static_cast<size_t>(row[i] < 0 ? 0 : row[i]) * (DSA_DIM * 2) + dc * 128 + p * 16,
                         row[i] >= 0 ? 16u : 0u);
            }
          };
          if (vals) {
            // a stage is handed over once the next tile's copies are on their way
            if (!(ok = wait_v(gg, u == 0))) break;
#pragma unroll
            for (int c = 0; c < VC; ++c) copy(vst + (gg % NV) * (VC * CH) + c * CH, 4 * half + c);
            cp_async_commit();
            if (u > 0) {
              cp_async_wait<1>();
              done(&v_full[(gg - 1) % NV]);
            }
          } else {
            if (!(ok = wait_a(gg, 0))) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) copy(ast + c * CH, 4 * (half ^ 1) + c);
            cp_async_commit();
            if (!(ok = wait_a(gg, 1))) break;
#pragma unroll
            for (int c = 2; c < AC + 1; ++c) copy(ast + c * CH, c < 4 ? 4 * (half ^ 1) + c : 8);
            cp_async_commit();
            cp_async_wait<1>();
            done(&a_full[0]);
            cp_async_wait<0>();
            done(&a_full[1]);
          }
        }
        if (vals) {
          cp_async_wait<0>();
          if (ok) done(&v_full[(g + n - 1) % NV]);
        }
      }
      g += n;
    }
    cp_async_wait<0>();                              // nothing in flight when the CTA retires
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Merge of the parts of queries whose tiles lie on several pairs: pair p holds
// the first part of query desc[2p + 1] in part 2p + 1, the pairs after it the
// others in parts 2(p + i), where desc[2(p + i)] is that query again.
//   LSE = ln sum_i exp(LSE_i),  O = sum_i exp(LSE_i - LSE) O_i.
// grid (pairs, H / 4): 4 heads a CTA, a float4 of one head's output a thread.
constexpr int MT = 512;
__global__ void __launch_bounds__(MT) attend_merge_kernel(const int32_t* desc, const float* o_part,
                                                          const float* l_part, int H, __nv_bfloat16* out,
                                                          float* lse) {
  pdl_wait();
  const int p = blockIdx.x, pairs = gridDim.x;
  const int q = desc[2 * p + 1];
  if (q < 0) return;
  int n = 1;
  while (p + n < pairs && desc[2 * (p + n)] == q) ++n;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 7), c = threadIdx.x & 127;
  float m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, l_part[static_cast<size_t>(2 * (p + i) + (i == 0)) * H + h]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float tot = 0.f;
  const float m_eff = m == -INFINITY ? 0.f : m;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const size_t at = static_cast<size_t>(2 * (p + i) + (i == 0)) * H + h;
    const float w = expf(l_part[at] - m_eff);
    const float4 v = reinterpret_cast<const float4*>(o_part + at * DSA_DIM_V)[c];
    tot += w;
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  const size_t qh = static_cast<size_t>(q) * H + h;
  reinterpret_cast<uint2*>(out + qh * DSA_DIM_V)[c] =
      make_uint2(bf16x2_bits(acc.x * inv, acc.y * inv), bf16x2_bits(acc.z * inv, acc.w * inv));
  if (c == 0) lse[qh] = tot == 0.f ? -INFINITY : m_eff + logf(tot);
}

constexpr int MAX_PAIRS = 74;
constexpr size_t DESC_OFF = 256;
constexpr size_t L_OFF = DESC_OFF + 2 * MAX_PAIRS * 4 + 176;      // 1024
static_assert(L_OFF % 256 == 0, "aligned");

template <bool KV8, bool IDX>
cudaError_t launch(const AttendArgs& a, int pairs, cudaStream_t st) {
  static std::atomic<bool> done[64];
  auto kernel = attend_kernel<KV8, IDX>;
  const cudaError_t e = set_once_per_device(done, [kernel] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  if (e != cudaSuccess) return e;
  kernel<<<2 * pairs, THREADS, SMEM_BYTES, st>>>(a);
  return cudaGetLastError();
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
  cudaError_t e = idx ? launch<true, true>(a, pairs, st)
                      : (kv_scales ? launch<true, false>(a, pairs, st) : launch<false, false>(a, pairs, st));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(H / 4), 1);
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
