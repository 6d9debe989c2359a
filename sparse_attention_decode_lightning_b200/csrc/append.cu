// Latent-cache append: the rows that the attention calls read are written here,
// the position part rotated on the way.  Token t of sequence b sits at position
// p = q_vis[t] - 1 and its row is
//   [ kv[t, 0:512] | rot(k_pe[t, 0:64]) ],
//   rot: (x, y) -> (x cos(a) - y sin(a), y cos(a) + x sin(a)),  a = p * inv_freq[i],
// with (x, y) = elements (i, i + 32), or (2i, 2i + 1) when interleaved.
//
// bf16 cache: the row rounded once.  e4m3 cache: the tokens of a block share
// one scale s = 2^e, e the smallest with amax <= 448 * 2^e in [-40, 40]; a
// block that already holds tokens keeps s = max(old, needed) and, when that
// grows, its codes are rescaled by old / s (a power of two, so a code changes
// only where it falls into e4m3's subnormals).
//
// The angle: p * inv_freq exceeds what fp32 resolves for far positions (1e6
// rad has a spacing of 1/16).  A lane keeps its turns a position, modulo 1, as a
// fraction of 2^64; p times that wraps as the angle does, and its upper half is
// the angle to 2^-32 of a turn.
//
// Bound: bytes (1152 read, 576 or 1152 written a token).  A run, the new rows of one
// block, is short, up to four rows, which one warp takes, or long, which all warps of
// the CTA share.  The kernel made for the sort that the batch has more of holds its
// rows in registers between the maximum and the rounding, up to four a warp, so a row
// is read once and all its loads are under way at once; rows of the other sort, and of
// blocks of more than 64 tokens, are read twice.
//
// Mixed batches (us of the GPU's time, blocks of 64): 512 single tokens 7.1, a chunk of
// 1024 9.8, both in one call 14.3; 64 single tokens 4.0, eight chunks of 4000 20.8, both
// 20.8.  One warp a run, or all warps a run, for the whole batch by its average length
// took 45.8 and 82.8.
//
// Measured: 32,000 tokens of eight prompts into blocks of 64, e4m3: 24.7 us, 2.3 TB/s,
// 2.9 times its bytes.  Two CTAs fit an SM, since the rows take the registers, so
// there are two rounds of about 10 us, each a chain of loads (offsets, position,
// page, rows) and one exchange of the maximum; sending the rows to L2 ahead of the
// chain made it 27.3 us.  8,000 tokens, bf16: 5.9 us of the GPU's time, 10.9 us with
// the call.  A single token: 3.2 us of the GPU's, 12 us with the call.
#include "common.cuh"
#include "internal.h"

#include <cuda_fp8.h>

namespace dsa {
namespace {

constexpr int MAX_G = 64;                  // rows of the token array a CTA looks for run starts in
constexpr int EXP_LIMIT = 40;
constexpr int KEEP = 4;                    // rows of a run that a warp holds in registers

struct AppendArgs {
  const __nv_bfloat16* kv;
  const __nv_bfloat16* k_pe;
  int64_t ld_kv, ld_pe;                    // row strides in elements
  const float* inv_freq;
  const int32_t* page_table;
  const int32_t* q_offsets;
  const int32_t* q_vis;
  uint8_t* pool;
  float* scales;
  uint32_t* err;
  int max_pages, B, T, num_pages, page_shift, block_shift, G, interleaved;
};

// 16 latent values (lane's 16 consecutive dims) and one rotated pair of a row
struct Row {
  uint4 a, b;
  float x, y;
};

// turns a position modulo 1, in 2^-64; a frequency that is no number has no angle
struct Freq {
  uint64_t step;
  float bad;                               // 0, or NaN
};

__device__ __forceinline__ Freq turns_of(float inv_freq) {
  Freq f;
  double t = static_cast<double>(inv_freq) * 0.15915494309189535;
  f.bad = inv_freq - inv_freq;
  t -= rint(t);                            // [-1/2, 1/2]
  f.step = f.bad == 0.f ? static_cast<uint64_t>(__double2ll_rn(t * 9223372036854775808.0)) << 1 : 0;
  return f;
}

__device__ __forceinline__ Row load_row(const AppendArgs& A, int t, int lane) {
  Row r;
  const uint4* src = reinterpret_cast<const uint4*>(A.kv + static_cast<int64_t>(t) * A.ld_kv) + 2 * lane;
  r.a = __ldg(src);
  r.b = __ldg(src + 1);
  const __nv_bfloat16* pe = A.k_pe + static_cast<int64_t>(t) * A.ld_pe;
  r.x = __bfloat162float(pe[A.interleaved ? 2 * lane : lane]);
  r.y = __bfloat162float(pe[A.interleaved ? 2 * lane + 1 : lane + 32]);
  return r;
}

__device__ __forceinline__ void rotate(Row& r, int pos, const Freq& f) {
  const int32_t turns = static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * f.step) >> 32);
  float s, c;
  sincospif(fmaf(static_cast<float>(turns), 0x1p-31f, f.bad), &s, &c);
  const float x = r.x;
  r.x = x * c - r.y * s;
  r.y = r.y * c + x * s;
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// |v| of a finite value, 0 of any other: what counts for a block's scale
__device__ __forceinline__ float mag(float v) {
  const float a = fabsf(v);
  return a <= 3.4028235e38f ? a : 0.f;
}

__device__ __forceinline__ float mag4(uint4 v) {
  return fmaxf(fmaxf(fmaxf(mag(lo_f(v.x)), mag(hi_f(v.x))), fmaxf(mag(lo_f(v.y)), mag(hi_f(v.y)))),
               fmaxf(fmaxf(mag(lo_f(v.z)), mag(hi_f(v.z))), fmaxf(mag(lo_f(v.w)), mag(hi_f(v.w)))));
}

__device__ __forceinline__ uint32_t pair_bits(uint32_t m, uint32_t w) {
  return max(max(m, (w << 16) & 0x7FFF0000u), w & 0x7FFF0000u);
}

// a lane's largest magnitude of a row, and whether all its values are finite:
// the magnitudes compare as integers, and what is not finite as the largest
__device__ __forceinline__ float lane_amax(const Row& r, bool* finite) {
  uint32_t m = max(__float_as_uint(fabsf(r.x)), __float_as_uint(fabsf(r.y)));
  m = pair_bits(pair_bits(pair_bits(pair_bits(m, r.a.x), r.a.y), r.a.z), r.a.w);
  m = pair_bits(pair_bits(pair_bits(pair_bits(m, r.b.x), r.b.y), r.b.z), r.b.w);
  *finite = m < 0x7F800000u;
  if (*finite) return __uint_as_float(m);
  return fmaxf(fmaxf(mag4(r.a), mag4(r.b)), fmaxf(mag(r.x), mag(r.y)));
}

__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));   // m >= 0
}

// smallest e in [-40, 40] with amax <= 448 * 2^e = 1.75 * 2^(e + 8)
__device__ __forceinline__ int needed_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return -EXP_LIMIT;
  const int k = static_cast<int>(u >> 23) - 127;          // a subnormal amax is far below the limit
  const int e = k - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(EXP_LIMIT, max(-EXP_LIMIT, e));
}

// v -> e4m3 code, round to nearest even; finite values saturate at 448, the
// others become the NaN code
__device__ __forceinline__ uint32_t f8(float v) {
  const float a = fabsf(v);
  if (!(a <= 3.4028235e38f)) return 0x7Fu;
  return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t f8_div4(uint32_t w0, uint32_t w1, float s) {
  return f8(__fdiv_rn(lo_f(w0), s)) | (f8(__fdiv_rn(hi_f(w0), s)) << 8) |
         (f8(__fdiv_rn(lo_f(w1), s)) << 16) | (f8(__fdiv_rn(hi_f(w1), s)) << 24);
}

// four values times inv, a power of two: scaling is exact but for subnormals, as
// the division would be
__device__ __forceinline__ uint32_t f8x4(uint32_t w0, uint32_t w1, float inv, bool finite) {
  const float a = lo_f(w0) * inv, b = hi_f(w0) * inv, c = lo_f(w1) * inv, d = hi_f(w1) * inv;
  if (finite)
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
  return f8(a) | (f8(b) << 8) | (f8(c) << 16) | (f8(d) << 24);
}

__device__ __forceinline__ void store_e4m3(const AppendArgs& A, int64_t slot, const Row& w, float inv, bool finite, int lane) {
  uint8_t* dst = A.pool + slot * DSA_DIM;
  reinterpret_cast<uint4*>(dst)[lane] = make_uint4(f8x4(w.a.x, w.a.y, inv, finite), f8x4(w.a.z, w.a.w, inv, finite),
                                                   f8x4(w.b.x, w.b.y, inv, finite), f8x4(w.b.z, w.b.w, inv, finite));
  dst[DSA_DIM_V + (A.interleaved ? 2 * lane : lane)] = static_cast<uint8_t>(f8(w.x * inv));
  dst[DSA_DIM_V + (A.interleaved ? 2 * lane + 1 : lane + 32)] = static_cast<uint8_t>(f8(w.y * inv));
}

__device__ __forceinline__ float f8_value(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  return f8(f8_value(w & 0xFFu) * ratio) | (f8(f8_value((w >> 8) & 0xFFu) * ratio) << 8) |
         (f8(f8_value((w >> 16) & 0xFFu) * ratio) << 16) | (f8(f8_value(w >> 24) * ratio) << 24);
}

// A run: the rows of one sequence that fall into one block of the cache
struct Run {
  int t, n;            // first row of the token array, rows
  int pos;             // position of the first row
  int vis0;            // q_vis expected at row t
  int64_t slot;        // pool row of the first row
};

// run that starts at row t, or n = 0
__device__ __forceinline__ Run find_run(const AppendArgs& A, const int* off, int t) {
  Run r = {t, 0, 0, 0, 0};
  if (t < off[0] || t >= off[A.B]) return r;              // rows outside every sequence stay as they are
  int lo = 0, hi = A.B;                                   // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  const int f = off[lo];
  if (f < 0 || f > t || off[lo + 1] > A.T) {              // offsets that are none: nothing is known of their rows
    raise_error(A.err, DEVERR_BOUNDS);
    return r;
  }
  const int v0 = A.q_vis[f];
  const int v = A.q_vis[t];
  if (v0 <= 0) {                                          // a padded sequence
    if (v != 0) raise_error(A.err, DEVERR_BOUNDS);
    return r;
  }
  const int64_t pos = static_cast<int64_t>(v0) - 1 + (t - f);
  const int bm = (1 << A.block_shift) - 1;
  if (t != f && (pos & bm) != 0) return r;                // belongs to the run before
  const int64_t page = pos >> A.page_shift;
  const int n = min(off[lo + 1] - t, bm + 1 - static_cast<int>(pos & bm));
  const int pg = page < A.max_pages ? A.page_table[static_cast<size_t>(lo) * A.max_pages + page] : -1;
  if (pg < 0 || pg >= A.num_pages) {
    // nothing to say where every row of the run is padding
    for (int i = 0; i < n; ++i)
      if (A.q_vis[t + i] != 0) {
        raise_error(A.err, DEVERR_BOUNDS);
        break;
      }
    return r;
  }
  r.n = n;
  r.pos = static_cast<int>(pos);
  r.vis0 = r.pos + 1;
  r.slot = (static_cast<int64_t>(pg) << A.page_shift) + (pos & ((1 << A.page_shift) - 1));
  return r;
}

// The rows of a run, bf16 cache: as they are, the position part rotated; by one warp
__device__ __forceinline__ void append_bf16(const AppendArgs& A, const Run& r, const Freq& freq, int lane) {
  for (int i = 0; i < r.n; ++i) {
    const int v = A.q_vis[r.t + i];
    if (v != r.vis0 + i) {
      if (v != 0 && lane == 0) raise_error(A.err, DEVERR_BOUNDS);
      continue;
    }
    Row w = load_row(A, r.t + i, lane);
    rotate(w, r.pos + i, freq);
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(A.pool) + (r.slot + i) * DSA_DIM;
    reinterpret_cast<uint4*>(dst)[2 * lane] = w.a;
    reinterpret_cast<uint4*>(dst)[2 * lane + 1] = w.b;
    dst[DSA_DIM_V + (A.interleaved ? 2 * lane : lane)] = __float2bfloat16_rn(w.x);
    dst[DSA_DIM_V + (A.interleaved ? 2 * lane + 1 : lane + 32)] = __float2bfloat16_rn(w.y);
  }
}

// The rows of a run, e4m3 cache, by W warps (1, or all of the CTA's, which then meet
// at barriers): this is warp wg of them.  HOLD: a warp holds up to KEEP rows in
// registers between the maximum and the rounding; else, and where there are more,
// they are read twice.  wmax: a word for each of the W.
template <int W, bool HOLD>
__device__ __forceinline__ void append_e4m3(const AppendArgs& A, const Run& r, const Freq& freq, int wg, int lane, float* wmax) {
  const int held = r.pos & ((1 << A.block_shift) - 1);       // tokens the block holds already
  float* sp = A.scales + (r.slot >> A.block_shift);
  const float old = held ? *sp : 0.f;
  float m = 0.f;
  bool any = false;
  Row keep[KEEP];
  uint32_t kept = 0, odd = 0;                                // rows in registers; of them not finite in this lane
  const bool held_back = HOLD && (W == 1 || r.n <= KEEP * W);   // every row stays in registers; one warp takes no more
  if (held_back) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int i = wg + j * W;
      if (i >= r.n) break;
      const int v = A.q_vis[r.t + i];
      if (v == r.vis0 + i) {
        kept |= 1u << j;
        keep[j] = load_row(A, r.t + i, lane);
      } else if (v != 0 && lane == 0) {
        raise_error(A.err, DEVERR_BOUNDS);
      }
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (kept >> j & 1u) {
        rotate(keep[j], r.pos + wg + j * W, freq);
        bool finite;
        m = fmaxf(m, lane_amax(keep[j], &finite));
        odd |= finite ? 0u : 1u << j;
      }
    any = kept != 0;
  } else {
    for (int i = wg; i < r.n; i += W) {
      const int v = A.q_vis[r.t + i];
      if (v != r.vis0 + i) {
        if (v != 0 && lane == 0) raise_error(A.err, DEVERR_BOUNDS);
        continue;
      }
      any = true;
      Row w = load_row(A, r.t + i, lane);
      rotate(w, r.pos + i, freq);
      bool finite;
      m = fmaxf(m, lane_amax(w, &finite));
    }
  }
  m = warp_max(m);
  if constexpr (W > 1) {
    if (lane == 0) wmax[wg] = any ? m : -1.f;
    __syncthreads();
    m = -1.f;
#pragma unroll
    for (int i = 0; i < W; ++i) m = fmaxf(m, wmax[i]);
    any = m >= 0.f;
    __syncthreads();                                         // wmax is free, every thread holds `old`
  }
  if (!any) return;                                          // nothing but padding
  float s = exp2f(static_cast<float>(needed_exp(m)));
  const bool old_ok = old >= 0x1p-40f && old <= 0x1p40f;
  if (held && !old_ok && lane == 0 && wg == 0) raise_error(A.err, DEVERR_BOUNDS);
  if (held && old_ok) s = fmaxf(s, old);
  __syncwarp();
  if (lane == 0 && wg == 0) *sp = s;
  if (held && old_ok && s > old) {
    const float ratio = __fdiv_rn(old, s);
    uint4* base = reinterpret_cast<uint4*>(A.pool + (r.slot - held) * DSA_DIM);
    for (int i = wg * 32 + lane; i < held * (DSA_DIM / 16); i += 32 * W) {
      uint4 c = base[i];
      c = make_uint4(rescale4(c.x, ratio), rescale4(c.y, ratio), rescale4(c.z, ratio), rescale4(c.w, ratio));
      base[i] = c;
    }
  }
  const float inv = __fdiv_rn(1.f, s);                       // exact where s is a power of two; an old scale may be none
  const bool exact = (__float_as_uint(s) & 0x7FFFFFu) == 0;
  if (held_back && exact) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (kept >> j & 1u) store_e4m3(A, r.slot + wg + j * W, keep[j], inv, !(odd >> j & 1u), lane);
  } else {
    for (int i = wg; i < r.n; i += W) {
      if (A.q_vis[r.t + i] != r.vis0 + i) continue;
      Row w = load_row(A, r.t + i, lane);
      rotate(w, r.pos + i, freq);
      if (exact) {
        bool finite;
        lane_amax(w, &finite);
        store_e4m3(A, r.slot + i, w, inv, finite, lane);
      } else {
        uint8_t* dst = A.pool + (r.slot + i) * DSA_DIM;
        reinterpret_cast<uint4*>(dst)[lane] = make_uint4(f8_div4(w.a.x, w.a.y, s), f8_div4(w.a.z, w.a.w, s),
                                                         f8_div4(w.b.x, w.b.y, s), f8_div4(w.b.z, w.b.w, s));
        dst[DSA_DIM_V + (A.interleaved ? 2 * lane : lane)] = static_cast<uint8_t>(f8(__fdiv_rn(w.x, s)));
        dst[DSA_DIM_V + (A.interleaved ? 2 * lane + 1 : lane + 32)] = static_cast<uint8_t>(f8(__fdiv_rn(w.y, s)));
      }
    }
  }
}

// A CTA takes the runs that start in its G rows: short ones (decode, verify steps,
// small blocks) a warp each, long ones with all warps together, whatever the batch
// mixes.  LONG: made for long runs, whose rows its 16 warps hold, 64 registers a
// thread; else for short ones (bf16: runs of one row), which a warp holds alone.  The
// other sort's rows are read twice, so that they take no registers from the first.
template <bool KV8, bool LONG>
__global__ void __launch_bounds__(LONG ? 512 : 256, LONG ? 2 : 1) latent_append_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int WARPS = LONG ? 16 : 8, THREADS = 32 * WARPS;
  __shared__ int off[DSA_MAX_BATCH + 1];
  __shared__ Run runs[MAX_G];                        // short ones from the front, long ones from the end
  __shared__ int n_short, n_long;
  __shared__ float wmax[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();                                     // an attention that follows sets itself up meanwhile
  if (tid == 0) n_short = n_long = 0;
  for (int i = tid; i <= A.B; i += THREADS) off[i] = A.q_offsets[i];
  __syncthreads();
  if (tid < A.G) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * A.G + tid;
    if (t < A.T) {
      const Run r = find_run(A, off, static_cast<int>(t));
      if (r.n > KEEP) runs[MAX_G - 1 - atomicAdd(&n_long, 1)] = r;   // any order: runs are independent
      else if (r.n > 0) runs[atomicAdd(&n_short, 1)] = r;
    }
  }
  __syncthreads();
  const Freq freq = turns_of(A.inv_freq[lane]);
  if constexpr (KV8) {
    for (int k = MAX_G - 1; k > MAX_G - 1 - n_long; --k) {
      const Run r = runs[k];
      append_e4m3<WARPS, LONG>(A, r, freq, warp, lane, wmax);
    }
    for (int k = warp; k < n_short; k += WARPS) {
      const Run r = runs[k];
      append_e4m3<1, !LONG>(A, r, freq, 0, lane, nullptr);
    }
  } else {
    for (int k = warp; k < n_short; k += WARPS) append_bf16(A, runs[k], freq, lane);
  }
}

}  // namespace

cudaError_t launch_latent_append(const __nv_bfloat16* kv, int64_t ld_kv, const __nv_bfloat16* k_pe,
                                 int64_t ld_pe, const float* inv_freq, int interleaved,
                                 const int32_t* page_table, int max_pages, const int32_t* q_offsets,
                                 const int32_t* q_vis, int B, int T, void* pool, float* scales,
                                 int num_pages, int page_size, int scale_block, uint32_t* err,
                                 cudaStream_t st) {
  AppendArgs A = {};
  A.kv = kv;
  A.k_pe = k_pe;
  A.ld_kv = ld_kv;
  A.ld_pe = ld_pe;
  A.inv_freq = inv_freq;
  A.page_table = page_table;
  A.q_offsets = q_offsets;
  A.q_vis = q_vis;
  A.pool = static_cast<uint8_t*>(pool);
  A.scales = scales;
  A.err = err;
  A.max_pages = max_pages;
  A.B = B;
  A.T = T;
  A.num_pages = num_pages;
  while ((1 << A.page_shift) < page_size) ++A.page_shift;
  while (scales && (1 << A.block_shift) < scale_block) ++A.block_shift;   // bf16: runs of one row
  A.interleaved = interleaved;
  // rows a CTA looks for run starts in: enough CTAs to fill the GPU four deep
  const int fill = 4 * device_sm_count();
  A.G = T / fill < 1 ? 1 : (T / fill > MAX_G ? MAX_G : T / fill);
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(T) + A.G - 1) / A.G);
  // The average rows a sequence say which sort of runs the batch has more of; either
  // kernel takes both.
  if (!scales) latent_append_kernel<false, false><<<grid, 256, 0, st>>>(A);
  else if (T <= static_cast<int64_t>(KEEP) * B || scale_block <= KEEP) latent_append_kernel<true, false><<<grid, 256, 0, st>>>(A);
  else latent_append_kernel<true, true><<<grid, 512, 0, st>>>(A);
  return cudaGetLastError();
}

}  // namespace dsa
