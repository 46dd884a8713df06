// A chunk of new tokens into the three-segment cache: byte for byte what as many appends
// write ("TogetherAI开源OSCAR" (ModelScope), section "OSCAR的设计": new tokens enter the BF16
// recent window, the oldest are rotated, clipped, quantised and packed).
//
// extend_history_kernel takes 128 history tokens of one kv head, K or V, at a time, whatever
// requests they are of, each from the ring or from the new rows:
//   x~ = k R        128 x 128 x 128 on tcgen05, R as two bf16 parts, the small one's products
//                   first; a token is a row of the accumulator, so a TMEM lane, so a thread;
//   min, max, code  the thread's 128 values, from TMEM twice: no exchange between lanes.
// A value's code is decided from x~ where the decision holds for every x within the error
// bound below.  Where it does not (1 token in 20 with thresholds at the 0.9 quantile, a value
// or an end of the range of each), the warp takes those values in turn by a compensated product
// (four at a time), whose bound leaves nearly nothing open; a token that is still open goes the
// append's way (quantize_group_warp): every byte is that of fp32_rn(k . R).
//
// Error of x~, with S = |k|_2 max_j |R_:j|_2 >= sum |k_i R_ij| and u = 2^-24: products are exact;
// one product step adds 16 of them to the accumulator, each of the 17 terms cut by at most one
// ulp of the largest and the result by one of itself, 36 u S; eight steps with R1 and eight with
// R2 before (2^-8 of that) 290 u S; what R1 + R2 leave of R 2^-18 S = 64 u S; x's own rounding
// u S: 355 u S < 0x1.7p-16 S.
//
// 8192 tokens of 8 kv heads: 37 us, of which the floor (k and v read once, 72 bytes a token-head written) is 5.7.  Half
// of it is latency and set-up -- a group of warps has two tiles, 10 us the first -- and 8 to 15 us are open values, most in
// the head whose tokens differ most in length, whose CTAs are the last.
//
// Four groups of four warps per CTA take tiles in turn, each with a tile of k in shared memory
// and an accumulator: what a group waits for (its copy, its products, rows of R for an open
// value), the others' decisions cover.
#include <atomic>

#include "append_device.cuh"
#include "chunk.h"
#include "quant_device.cuh"
#include "tcgen05_device.cuh"

namespace oscar {
namespace {

using namespace paged;

constexpr int EX_ROWS = 128;                   // history tokens of a tile
constexpr int EX_GROUPS = 4;                   // groups of four warps
constexpr int EX_THREADS = EX_GROUPS * EX_ROWS;
constexpr float EX_MMA_ERR = 0x1.7p-16f;

struct alignas(1024) ExtendSmem {
  alignas(1024) uint8_t r[2][TILE_BYTES];                   // R2^T, R1^T: two halves of 64 inputs, [128 outputs][128 B] swizzled
  alignas(1024) uint8_t k[EX_GROUPS][TILE_BYTES];           // tiles of tokens, likewise
  const uint16_t* src[EX_GROUPS][EX_ROWS];                  // where a tile's rows are, null: none
  float x[EX_GROUPS * 4][D];                                // a token that its warp decides
  uint64_t done[EX_GROUPS];                                 // the accumulator's products are done
  uint32_t tmem;
};
static_assert(sizeof(ExtendSmem) + 1024 <= 232448, "shared memory of a CTA");

// Byte offset of 16 bytes (8 channels) of a row in a swizzled tile.
__device__ __forceinline__ uint32_t tile_at(int row, int part) {
  return (part >> 3) * (TILE_BYTES / 2) + row * 128 + (((part & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(EX_ROWS) : "memory");
}
// A barrier of the group that says whether all its threads answer yes.
__device__ __forceinline__ bool group_all(int group, bool mine) {
  int all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.b32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(static_cast<int>(mine)), "r"(group + 1), "n"(EX_ROWS)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float fma_sat(float a, float b, float c) {
  float d;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint16_t half_bits(float x) { return __half_as_ushort(__float2half_rn(x)); }

// The group's scale, zero and code steps from its extremes, each known to lie between two (clipped)
// values; false where they are open.
struct Range {
  float mn_lo, mn_hi, mx_lo, mx_hi;
};
struct Grid {
  uint16_t s_bits, z_bits;
  float a, b, margin;   // code = rint(3 sat(a x + b)), where 3 sat() is not within margin of a half
};
__device__ __forceinline__ bool grid_of(const Range& r, float e, Grid& g) {
  g.z_bits = half_bits(r.mn_lo);
  const float s = scale_of(r.mx_lo, r.mn_hi);
  g.s_bits = half_bits(s);
  const bool sure = g.z_bits == half_bits(r.mn_hi) && s == scale_of(r.mx_hi, r.mn_lo);
  if (s == 0.0f) {   // every code is 0
    g.a = g.b = 0.0f;
    g.margin = 0.25f;
    return sure;
  }
  // q = (x - z) / s: the reciprocal and its third are off by 2^-22, b's rounding by |z / s| 2^-24,
  // the quotient of the definition by 2^-22 of q
  const float z = __half2float(__ushort_as_half(g.z_bits)), rs = rcp_approx(s);
  g.a = rs * (1.0f / 3.0f);
  g.b = -z * g.a;
  g.margin = fmaf(fmaf(fabsf(z), 0x1p-21f, 1.001f * e), rs, 0x1p-18f);
  // values beyond the thresholds take the code of the threshold: 3 and 0, so that they need no clip
  return sure && (r.mx_lo - z) * rs > 2.5f + g.margin && (r.mn_hi - z) * rs < 0.5f - g.margin && g.margin < 0.25f;
}

// The compensated product of warp_dot2 by eight lanes, 16 terms each: bounds lo <= fp32_rn(exact) <= hi.  The error
// terms are at most 19 u S in all (a product's u, a sum's u of what it has so far) and their own sum, 21 additions
// deep, is off by 21 u of that: 2^-39.4 S, within the 2^-36 S taken.  Each bound is rounded once, and to nearest as
// the exact sum is, so that the two are nearly always the same value.
__device__ __forceinline__ void dot2_of_eight(const uint4* k, const float4* r, float S, float& lo, float& hi) {
  uint4 kw[2];
  float4 rv[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) kw[j] = k[j];
#pragma unroll
  for (int j = 0; j < 4; ++j) rv[j] = __ldg(r + j);
  float s = 0.0f, c = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w0 = j & 1 ? kw[j >> 1].z : kw[j >> 1].x, w1 = j & 1 ? kw[j >> 1].w : kw[j >> 1].y;
    const float a[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xffff0000u), __uint_as_float(w1 << 16),
                        __uint_as_float(w1 & 0xffff0000u)};
    const float b[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p = __fmul_rn(a[i], b[i]), q = __fmaf_rn(a[i], b[i], -p);
      float e;
      two_sum_f(s, p, s, e);
      c = __fadd_rn(c, __fadd_rn(e, q));
    }
  }
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, s, off), c2 = __shfl_xor_sync(0xffffffffu, c, off);
    float e;
    two_sum_f(s, s2, s, e);
    c = __fadd_rn(c, __fadd_rn(c2, e));
  }
  const float E = __fmul_ru(S, 0x1p-36f);
  lo = __fadd_rn(s, __fsub_rd(c, E));
  hi = __fadd_rn(s, __fadd_ru(c, E));
}

constexpr float MAGIC = 12582912.0f;   // 1.5 2^23: adding it rounds to the nearest whole number

template <int GK>
__global__ void __launch_bounds__(EX_THREADS, 1)
    extend_history_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ExtendArgs A, int tiles,
                          int per_matrix) {
  extern __shared__ uint8_t ex_raw[];
  ExtendSmem& sm = *reinterpret_cast<ExtendSmem*>(ex_raw + (-smem_u32(ex_raw) & 1023u));
  constexpr int NG = D / GK;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int group = warp >> 2, r = threadIdx.x & (EX_ROWS - 1);
  const int matrix = blockIdx.x / per_matrix, part = blockIdx.x % per_matrix;
  const int head = matrix >> 1, which = matrix & 1;
  const size_t lh = (size_t)A.layer * c.Hkv + head;
  const float* Rt = (which ? c.rot_vt : c.rot_kt) + lh * D * D;
  const float tau = (which ? c.tau_v : c.tau_k)[lh], colnorm = c.rot_cn[(size_t)which * c.L * c.Hkv + lh];
  const uint16_t* fresh = (which ? A.v : A.k) + (size_t)head * D;
  const int64_t stride = which ? A.v_stride : A.k_stride;

  if (threadIdx.x == 0) {
    for (int g = 0; g < EX_GROUPS; ++g) mbar_init(&sm.done[g], 1);
    mbar_init_fence();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // R^T = R1 + R2 + d, written once at the cache's creation: before the grid's dependency
#pragma unroll 4
  for (int i = threadIdx.x; i < D * (D / 8); i += EX_THREADS) {
    const int n = i / (D / 8), p = i % (D / 8);
    const float4* src = reinterpret_cast<const float4*>(Rt + (size_t)n * D + 8 * p);
    const float4 f0 = src[0], f1 = src[1];
    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = f[2 * j], b = f[2 * j + 1];
      hi[j] = bf16x2(a, b);
      lo[j] = bf16x2(a - __uint_as_float(hi[j] << 16), b - __uint_as_float(hi[j] & 0xffff0000u));
    }
    *reinterpret_cast<uint4*>(sm.r[0] + tile_at(n, p)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(sm.r[1] + tile_at(n, p)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
  fence_async_smem();
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const int total = A.hist[A.n];
  // (few tiles go to CTAs of their own)
  const int step = EX_GROUPS * per_matrix, first = part + per_matrix * group;
  // Tile t: this thread looks its row up, then the group copies all rows, 16 bytes at a time.
  const uint16_t* src = nullptr;   // this thread's row
  uint8_t* dst = nullptr;          // its record, and its row there
  int row = 0;
  auto load = [&](int t) {
    const int i = t * EX_ROWS + r;
    src = nullptr;
    dst = nullptr;
    if (i < total) {
      int ri = 0, hi = A.n;
      while (hi - ri > 1) {
        const int mid = (ri + hi) >> 1;
        if (A.hist[mid] <= i) ri = mid; else hi = mid;
      }
      const int pos = A.h0[ri] + (i - A.hist[ri]), slot = A.slot[ri], at = pos - SINK;
      if (pos >= A.old[ri]) {
        src = fresh + (int64_t)(A.row0[ri] + (pos - A.old[ri])) * stride;
      } else {
        const int page = c.bf16_pt[(size_t)slot * BF16_PAGES_PER_REQ + 1 + (at % RECENT) / PAGE];
        if (page >= 0 && page < c.n_bf16_pages)
          src = bf16_row(c, A.layer, page, head, which, at % PAGE);
        else
          atomicOr(c.err, ERR_BF16_PAGE);
      }
      const int page = c.hist_pt[(size_t)slot * c.max_pages + at / PAGE];
      if (page >= 0 && page < c.n_int2_pages)
        dst = int2_record(c, A.layer, page, head);
      else
        atomicOr(c.err, ERR_INT2_PAGE);
      if (!src) dst = nullptr;
      row = at % PAGE;
    }
    sm.src[group][r] = src;
    group_sync(group);
#pragma unroll
    for (int u = 0; u < EX_ROWS * (D / 8) / EX_ROWS; ++u) {
      const int rw = u * (EX_ROWS / (D / 8)) + r / (D / 8), p = r % (D / 8);
      const uint16_t* s = sm.src[group][rw];
      cp_async16(sm.k[group] + tile_at(rw, p), s ? s + 8 * p : fresh, s != nullptr);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the landed tile's products into its accumulator
  auto multiply = [&]() {
    if ((warp & 3) != 0) return;
    tc_fence_after();
    const uint64_t k = desc_kmajor(smem_u32(sm.k[group]));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t w = desc_kmajor(smem_u32(sm.r[h]));
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint64_t off = ((s >> 2) * (TILE_BYTES / 2) + (s & 3) * 32) >> 4;
        mma_ss(128 * group, k + off, w + off, IDESC_QK, h > 0 || s > 0);
      }
    }
    mma_commit(&sm.done[group]);
  };
  // the bound S of this thread's row of a landed tile
  auto bound = [&]() {
    float sq = 0.0f;
#pragma unroll 4
    for (int p = 0; p < D / 8; ++p) {
      const uint4 v = *reinterpret_cast<const uint4*>(sm.k[group] + tile_at(r, p));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f0 = __uint_as_float(w[j] << 16), f1 = __uint_as_float(w[j] & 0xffff0000u);
        sq = __fmaf_ru(f0, f0, sq);
        sq = __fmaf_ru(f1, f1, sq);
      }
    }
    return __fmul_ru(__fsqrt_ru(__fmul_ru(sq, 1.0001f)), colnorm);
  };
  auto landed = [&]() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    fence_async_smem();
    tc_fence_before();
    group_sync(group);
  };

  bool ok = true;
  int count = 0;   // tiles of this group so far
  if (first < tiles) load(first);
  for (int t = first; t < tiles; t += step, ++count) {
    landed();
    multiply();
    const float S = bound();
    const uint16_t* const mine = src;
    uint8_t* const to = dst;
    const int place = row;
    // a wait that gave up is the group's, whose warps leave together; the tile is free
    ok = group_all(group, mbar_wait(&sm.done[group], count & 1));
    if (!ok) break;
    tc_fence_after();
    if (t + step < tiles) load(t + step);

    const uint32_t acc = (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 128 * group;
    const float e = __fmul_ru(S, EX_MMA_ERR);
    // The values that lanes have open, bit i of a lane's mask[h] channel ch0 + 32 h + i of its token, each to within
    // 2^-36 S and clipped: done(32 h + i, lo, hi) in its lane.  Four at a time, eight lanes each (one by one, every
    // value waited for a row of R and of k of its own).
    auto narrow = [&](uint32_t (&mask)[4], int ch0, auto done) {
#pragma unroll 1
      for (;;) {
        const int word = mask[0] ? 0 : mask[1] ? 1 : mask[2] ? 2 : 3;
        const uint32_t bits = mask[0] ? mask[0] : mask[1] ? mask[1] : mask[2] ? mask[2] : mask[3];
        const uint32_t open = __ballot_sync(0xffffffffu, bits != 0);
        if (!open) break;
        const int first = 32 * word + __ffs(bits) - 1;   // (of no use where none is open)
        uint32_t rest = open;
        int from = __ffs(open) - 1;   // the lane of these eight lanes' value
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (lane >> 3 == j && rest) from = __ffs(rest) - 1;
          rest &= rest - 1;
        }
        const int i = __shfl_sync(0xffffffffu, first, from);
        const auto* row = reinterpret_cast<const uint16_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), from));
        const float bound_of = __shfl_sync(0xffffffffu, S, from);
        float lo, hi;
        dot2_of_eight(reinterpret_cast<const uint4*>(row) + 2 * (lane & 7),
                      reinterpret_cast<const float4*>(Rt + (size_t)(ch0 + i) * D) + 4 * (lane & 7), bound_of, lo, hi);
        const int rank = __popc(open & ((1u << lane) - 1));
        lo = __shfl_sync(0xffffffffu, lo, 8 * (rank & 3));
        hi = __shfl_sync(0xffffffffu, hi, 8 * (rank & 3));
        if (bits != 0 && rank < 4) {
          done(first, clip_canon(lo, tau), clip_canon(hi, tau));
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (h == word) mask[h] &= mask[h] - 1;
        }
      }
    };
    // (Loops that stay loops: what is rare must not push what is not out of the instruction caches.  Arrays with a
    // running index are taken apart into selects.)
    Grid g[NG];
    bool sure = true;
#pragma unroll 1
    for (int n = 0; n < NG; ++n) {
      Grid gn;
      float mn = INFINITY, mx = -INFINITY;
#pragma unroll
      for (int h = 0; h < GK / 32; ++h) {
        uint32_t w[32];
        tmem_ld32(acc + n * GK + 32 * h, w);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          mn = min3(mn, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
          mx = max3(mx, __uint_as_float(w[i]), __uint_as_float(w[i + 1]));
        }
      }
      Range range{clip_canon(__fsub_rd(mn, e), tau), clip_canon(__fadd_ru(mn, e), tau), clip_canon(__fsub_rd(mx, e), tau),
                  clip_canon(__fadd_ru(mx, e), tau)};
      bool known = grid_of(range, e, gn) || !to;
      if (!__all_sync(0xffffffffu, known)) {
        // an end that is open: the values that may be it (the others lie inside), one after another
        const bool low = range.mn_lo != range.mn_hi, high = range.mx_lo != range.mx_hi;
        const float below = low && !known ? __fadd_ru(mn, 2.0f * e) : -INFINITY, above = high && !known ? __fsub_rd(mx, 2.0f * e) : INFINITY;
        float lo0 = INFINITY, lo1 = INFINITY, hi0 = -INFINITY, hi1 = -INFINITY;
        uint32_t open[4] = {0, 0, 0, 0};
#pragma unroll 1
        for (int h = 0; h < GK / 32; ++h) {
          uint32_t w[32], mask = 0;
          tmem_ld32(acc + n * GK + 32 * h, w);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            mask |= __uint_as_float(w[i]) <= below || __uint_as_float(w[i]) >= above ? 1u << i : 0u;
#pragma unroll
          for (int j = 0; j < GK / 32; ++j)
            if (j == h) open[j] = mask;
        }
        narrow(open, n * GK, [&](int, float lo, float hi) {
          lo0 = fminf(lo0, lo), lo1 = fminf(lo1, hi);
          hi0 = fmaxf(hi0, lo), hi1 = fmaxf(hi1, hi);
        });
        if (!known) {
          if (low) range.mn_lo = lo0, range.mn_hi = lo1;
          if (high) range.mx_lo = hi0, range.mx_hi = hi1;
          known = grid_of(range, e, gn);
        }
      }
      sure = sure && known;
#pragma unroll
      for (int j = 0; j < NG; ++j)
        if (j == n) g[j] = gn;
    }
    uint32_t code[8];
    uint32_t close = 0;   // 32 channels with a value near a border
#pragma unroll 1
    for (int h = 0; h < 4; ++h) {
      Grid q = g[0];
      if (NG == 2 && h >= 2) q = g[NG - 1];
      uint32_t w[32], two[2];
      tmem_ld32(acc + 32 * h, w);
      tc_wait_ld();
      constexpr uint32_t MAGIC_SUM = 0x4B400000u * 0x55555555u;   // MAGIC's bits in every 2-bit place, modulo 2^32
      float off = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t bits = 0u - MAGIC_SUM;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 y = make_float2(fma_sat(__uint_as_float(w[16 * j + i]), q.a, q.b),
                                       fma_sat(__uint_as_float(w[16 * j + i + 1]), q.a, q.b));
          const float2 three = make_float2(3.0f, 3.0f);
          const float2 near = fma2(y, three, make_float2(MAGIC, MAGIC));
          const float2 whole = add2(near, make_float2(-MAGIC, -MAGIC));
          const float2 d = fma2(y, three, make_float2(-whole.x, -whole.y));
          off = max3(off, fabsf(d.x), fabsf(d.y));
          bits += (__float_as_uint(near.x) << (2 * i)) + (__float_as_uint(near.y) << (2 * i + 2));
        }
        two[j] = bits;
      }
      close |= off < 0.5f - q.margin ? 0u : 1u << h;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j == h) code[2 * j] = two[0], code[2 * j + 1] = two[1];
    }
    if (!to || !sure) close = 0;
    if (__any_sync(0xffffffffu, close != 0)) {
      uint32_t open[4] = {0, 0, 0, 0};
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        if (!__any_sync(0xffffffffu, close >> h & 1)) continue;
        Grid q = g[0];
        if (NG == 2 && h >= 2) q = g[NG - 1];
        uint32_t w[32], mask = 0;
        tmem_ld32(acc + 32 * h, w);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float y = fma_sat(__uint_as_float(w[i]), q.a, q.b), whole = fmaf(y, 3.0f, MAGIC) - MAGIC;
          mask |= fabsf(fmaf(y, 3.0f, -whole)) < 0.5f - q.margin ? 0u : 1u << i;
        }
        if (!(close >> h & 1)) mask = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j == h) open[j] = mask;
      }
      narrow(open, 0, [&](int i, float lo, float hi) {
        const Grid& q = NG == 2 && i >= GK ? g[NG - 1] : g[0];
        const float z = __half2float(__ushort_as_half(q.z_bits)), s = __half2float(__ushort_as_half(q.s_bits));
        const uint32_t c0 = code_of(lo, z, s), at = 2 * (i & 15);
        if (c0 != code_of(hi, z, s)) sure = false;
        const int word = i >> 4;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j == word) code[j] = (code[j] & ~(3u << at)) | c0 << at;
      });
    }
    tc_fence_before();
    if (to && sure) {
      uint4* out = reinterpret_cast<uint4*>(to + (which ? V_CODES_OFF : K_CODES_OFF) + place * CODE_BYTES);
      out[0] = make_uint4(code[0], code[1], code[2], code[3]);
      out[1] = make_uint4(code[4], code[5], code[6], code[7]);
      uint32_t* meta = reinterpret_cast<uint32_t*>(to + (which ? v_meta_off_for(GK) : k_meta_off_for(GK)) +
                                                   place * meta_bytes_for(GK));
#pragma unroll
      for (int n = 0; n < NG; ++n) meta[n] = g[n].s_bits | (static_cast<uint32_t>(g[n].z_bits) << 16);
    }
    // the warp decides the tokens that are still open, one at a time
    for (uint32_t open = __ballot_sync(0xffffffffu, to && !sure); open; open &= open - 1) {
      const int from = __ffs(open) - 1;
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        uint32_t w[32];
        tmem_ld32(acc + 32 * h, w);
        tc_wait_ld();
        if (lane == from)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(&sm.x[warp][32 * h + i]) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      }
      __syncwarp();
      const float4 x = *reinterpret_cast<const float4*>(&sm.x[warp][4 * lane]);
      const auto* s = reinterpret_cast<const uint16_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), from));
      auto* rec = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), from));
      const int slot = __shfl_sync(0xffffffffu, place, from);
      const float sb = __shfl_sync(0xffffffffu, S, from), eb = __shfl_sync(0xffffffffu, e, from);
      const uint2 kw = reinterpret_cast<const uint2*>(s)[lane];
      const float4 k4 = make_float4(__uint_as_float(kw.x << 16), __uint_as_float(kw.x & 0xffff0000u),
                                    __uint_as_float(kw.y << 16), __uint_as_float(kw.y & 0xffff0000u));
      const GroupCode code_of_warp = quantize_group_warp<GK>(x, make_float4(eb, eb, eb, eb),
                                                             make_float4(sb, sb, sb, sb), tau, k4, Rt);
      store_group_code_t<GK>(rec, which, slot, code_of_warp);
      __syncwarp();
    }
  }
  if (!ok) {
    if (lane == 0) atomicOr(c.err, ERR_TIMEOUT);
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(0u) : "memory");
  }
}

// The new tokens that the sink or the recent window holds: 16 lanes a row of one kv head, K or V.
constexpr int EB_THREADS = 256;
__global__ void __launch_bounds__(EB_THREADS)
    extend_bf16_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ExtendArgs A) {
  grid_dep_launch();
  grid_dep_wait();   // the history kernel has read what the ring held
  const int64_t unit = ((int64_t)blockIdx.x * EB_THREADS + threadIdx.x) / (D / 8);   // (row, kv head, K or V)
  const int part = threadIdx.x % (D / 8), which = static_cast<int>(unit & 1);
  const int head = static_cast<int>((unit >> 1) % c.Hkv), i = static_cast<int>((unit >> 1) / c.Hkv);
  // row i of those that stay: of each request its sink tokens and its last ones, from tail on
  if (i >= A.rows[A.n]) return;
  int ri = 0, hi = A.n;
  while (hi - ri > 1) {
    const int mid = (ri + hi) >> 1;
    if (A.rows[mid] <= i) ri = mid; else hi = mid;
  }
  const int old = A.old[ri], sinks = max(0, SINK - old), at = i - A.rows[ri];
  const int kept = max(old, max(A.h1[ri], SINK));   // first new token that the window holds
  const int count = A.rows[ri + 1] - A.rows[ri];
  const int in_sink = min(sinks, count);
  const int pos = at < in_sink ? old + at : kept + (at - in_sink);
  const uint16_t* src = (which ? A.v + (int64_t)(A.row0[ri] + pos - old) * A.v_stride
                               : A.k + (int64_t)(A.row0[ri] + pos - old) * A.k_stride) + (size_t)head * D;
  const int page = c.bf16_pt[(size_t)A.slot[ri] * BF16_PAGES_PER_REQ + (pos < SINK ? 0 : 1 + (pos - SINK) % RECENT / PAGE)];
  if (page < 0 || page >= c.n_bf16_pages) {
    if (part == 0) atomicOr(c.err, ERR_BF16_PAGE);
    return;
  }
  reinterpret_cast<uint4*>(bf16_row(c, A.layer, page, head, which, pos % PAGE))[part] =
      reinterpret_cast<const uint4*>(src)[part];
}

template <int GK>
cudaError_t launch_history(const DevCache& c, const ExtendArgs& a, int sms, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(ExtendSmem)) + 1024;
  static std::atomic<unsigned> done;   // devices that have been set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(done.load() & (1u << dev))) {
    e = cudaFuncSetAttribute(extend_history_kernel<GK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 32) done.fetch_or(1u << dev);
  }
  // CTAs for each of the 2 Hkv matrices: one per SM in all, none without a tile
  const int tiles = (a.hist[a.n] + EX_ROWS - 1) / EX_ROWS, matrices = 2 * c.Hkv;
  const int fair = sms / matrices > 1 ? sms / matrices : 1, per_matrix = tiles < fair ? tiles : fair;
  return launch_dependent(extend_history_kernel<GK>, static_cast<unsigned>(matrices * per_matrix), EX_THREADS, bytes, s,
                          c, a, tiles, per_matrix);
}

}  // namespace

cudaError_t launch_extend_history(const DevCache& c, const ExtendArgs& a, int sms, cudaStream_t s) {
  return c.gk == 64 ? launch_history<64>(c, a, sms, s) : launch_history<128>(c, a, sms, s);
}

cudaError_t launch_extend_bf16(const DevCache& c, const ExtendArgs& a, cudaStream_t s) {
  const int64_t threads = (int64_t)a.rows[a.n] * c.Hkv * 2 * (D / 8);
  return launch_dependent(extend_bf16_kernel, static_cast<unsigned>((threads + EB_THREADS - 1) / EB_THREADS), EB_THREADS,
                          0, s, c, a);
}

}  // namespace oscar
