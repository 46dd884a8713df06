// Position rotation with append to a paged cache, and the 4-bit read-back.
//
// The row of every rotated head pairs channel i with j (i + dim / 2, or the
// neighbour of an interleaved pair) over the first dim channels:
//   y_i = x_i cos - x_j sin,   y_j = x_j cos + x_i sin,
// cosine and sine of position * frequency from the caller's fp32 table.  Every
// product and sum is rounded to fp32 by itself (no fused multiply-add) and the
// result once to bf16, so that a 4-bit code, which hangs on the exact value, is
// the same wherever the same formula is evaluated.
// The 4-bit cache holds, per token, kv head and group of 128 or 64 channels,
//   z = fp16(min x), s = fp16((max x - min x) / 15),
//   code = clamp(round_half_even((x - z) / s), 0, 15), 0 where s = 0,
// of the bf16 values that the BF16 cache would hold, saturated to +-65504 (the
// fp16 range of z) with NaN taken as 0; it stands for s code + z.
//
// A warp takes 16 head rows of a token, eight lanes a row, a lane both halves of its
// channel pairs: the rotation needs no exchange, and an access is 16 bytes a lane, whole
// sectors of eight lanes (two of 16 in one sector by turns: 66 against 58 us).  Bound by
// DRAM: BF16, 32K tokens of 32 + 8 heads in 120 us (6.9 TB/s); 4 bits, 16K tokens in 58 us
// (6.2 TB/s), with the quantiser's code rolled up, since four copies do not fit the
// instruction cache, and seven CTAs an SM (five: 100 against 91 us with the read-back).  A
// step of one token is a launch, 3.5 us on the GPU.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "paged_device.cuh"

namespace oscar {
namespace {

constexpr int APP_THREADS = 128;
constexpr int APP_ROWS = 4;                    // head rows per lane group in flight
constexpr int APP_HEADS = 4 * APP_ROWS;        // head rows per warp: four groups of 8 lanes

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t max_bf2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t neg_bf2(uint32_t a) { return a ^ 0x80008000u; }
// two fp32 operations in one instruction, each rounded by itself
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ uint32_t swap16(uint32_t a) { return __byte_perm(a, a, 0x1032); }

__device__ __forceinline__ int find_req(const PagedRows& r, int n, int row) {
  int lo = 0, hi = n;   // row0[lo] <= row < row0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (r.row0[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

// Page of position pos of request i, -1 (and the error bit) if its id is out of range.
__device__ __forceinline__ int64_t page_of(const PagedView& p, int i, int pos) {
  const int32_t page = p.table[(size_t)i * p.max_pages + pos / PAGE];
  if (page >= 0 && page < p.num_pages) return page;
  if (p.err) atomicOr(p.err, PAGED_ERR_PAGE);
  return -1;
}

// The rare paths are functions of their own: inlined for every row, they made the kernel
// wait for its instructions.
__device__ __forceinline__ float saturated(float x) {
  return x == x ? fminf(fmaxf(x, -65504.0f), 65504.0f) : 0.0f;
}
__device__ __forceinline__ float element(const uint4& x, int e) {
  const uint32_t w = e < 4 ? (e < 2 ? x.x : x.y) : (e < 6 ? x.z : x.w);
  return e & 1 ? bf_hi(w) : bf_lo(w);
}
// Codes of 8 channels by the definition.
__device__ __noinline__ uint32_t codes_exact(uint4 x, float s, float z) {
  uint32_t w = 0;
#pragma unroll 1
  for (int e = 7; e >= 0; --e) {
    const float t = rintf(__fdiv_rn(__fsub_rn(saturated(element(x, e)), z), s));
    const int code = s == 0.0f ? 0 : static_cast<int>(fminf(fmaxf(t, 0.0f), 15.0f));
    w = w << 4 | static_cast<uint32_t>(code);
  }
  return w;
}
// Least and greatest of 8 saturated channels.
__device__ __noinline__ float2 range_exact(uint4 x) {
  float2 r = make_float2(INFINITY, -INFINITY);
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    const float v = saturated(element(x, e));
    r.x = fminf(r.x, v);
    r.y = fmaxf(r.y, v);
  }
  return r;
}

// Codes of 8 finite channels within fp16 (four words of bf16 pairs) with scale s > 0 or
// s = 0 and zero z.  The quotient (x - z) / s, rounded as the definition has it, by one
// step of residual correction (Markstein, IBM J. Res. Dev. 34, 1990): t = d (1 / s) from an
// approximate reciprocal is within 15.5 (2^-23 + 2^-24) of it; e = d - t s is exact (t s has
// 35 bits, and what is left of d 14); t + e (1 / s) is within 2^-39 of the quotient before
// its one rounding, while no quotient of a fp32 number by one of 11 bits lies nearer than
// 2^-32 to the middle between two fp32 numbers from 1/4 to 16 (nor in it).  (Deciding the
// quotients near a half by a division took 18 % of the kernel: with 11-bit scales one warp
// in seven holds an exact tie.)  Magic: adding 1.5 2^23 rounds to the nearest integer, ties
// to even.
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&x)[4], float s, float z, bool wild) {
  constexpr float MAGIC = 12582912.0f;
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.0f) inv = 0.0f;
  const float2 zz = make_float2(-z, -z), ii = make_float2(inv, inv), ss = make_float2(-s, -s),
               mm = make_float2(MAGIC, MAGIC);
  // r's bits are those of MAGIC plus the code: weighted by 16^e they add up to the word
  // plus a constant
  uint32_t w = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 d = add2(make_float2(bf_lo(x[k]), bf_hi(x[k])), zz), t0 = mul2(d, ii);
    float2 t = fma2(fma2(t0, ss, d), ii, t0);
    t.x = fminf(fmaxf(t.x, 0.0f), 15.0f);
    t.y = fminf(fmaxf(t.y, 0.0f), 15.0f);
    const float2 r = add2(t, mm);
    w += (__float_as_uint(r.x) << (8 * k)) + (__float_as_uint(r.y) << (8 * k + 4));
  }
  if (wild) w = codes_exact(make_uint4(x[0], x[1], x[2], x[3]), s, z);
  return w;
}

// Quantise one head row held by 8 lanes, 16 channels each: chunks c[0] and c[1] of 8
// channels.  Writes the codes and, from the lane that holds a group's first chunk, {s, z}.
// Maxima and negated minima of a group travel as one bf16 pair.
template <int GK>
__device__ __forceinline__ void store_int4(uint8_t* rec, int which, int slot, const int (&c)[2],
                                           const uint32_t (&x)[2][4], bool ok) {
  constexpr int NG = D / GK;
  uint32_t top = 0;   // largest magnitude, NaN above infinity
  uint32_t mm[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) mm[g] = 0xff80ff80u;   // -infinity, twice
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t hi = x[u][0], lo = neg_bf2(x[u][0]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      top = __vmaxu2(top, x[u][k] & 0x7fff7fffu);
      if (k > 0) {
        hi = max_bf2(hi, x[u][k]);
        lo = max_bf2(lo, neg_bf2(x[u][k]));
      }
    }
    hi = max_bf2(hi, swap16(hi));
    lo = max_bf2(lo, swap16(lo));
    const uint32_t both = __byte_perm(hi, lo, 0x5410);
#pragma unroll
    for (int g = 0; g < NG; ++g) mm[g] = max_bf2(mm[g], NG == 1 || c[u] / (GK / 8) == g ? both : 0xff80ff80u);
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) mm[g] = max_bf2(mm[g], __shfl_xor_sync(0xffffffffu, mm[g], off));
  float mx[NG], mn[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    mx[g] = bf_lo(mm[g]);
    mn[g] = -bf_hi(mm[g]);
  }
  // values beyond fp16 (65280 is bf16's last below 65504) or NaN in the warp: once more, with care
  const bool wild = __any_sync(0xffffffffu, (top & 0xffffu) > 0x477fu || (top >> 16) > 0x477fu);
  if (wild) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      mn[g] = INFINITY;
      mx[g] = -INFINITY;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float2 v = range_exact(make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const bool in = NG == 1 || c[u] / (GK / 8) == g;
        mn[g] = fminf(mn[g], in ? v.x : INFINITY);
        mx[g] = fmaxf(mx[g], in ? v.y : -INFINITY);
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) {
        mn[g] = fminf(mn[g], __shfl_xor_sync(0xffffffffu, mn[g], off));
        mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], off));
      }
  }
  uint32_t sz[NG];   // {s, z}
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    // a / 15, rounded: the residual correction again, with the rounded reciprocal (where a
    // is so small that the residual is not exact, s is 0)
    const float a = __fsub_rn(mx[g], mn[g]), q = __fmul_rn(a, 1.0f / 15.0f);
    const __half2 both = __floats2half2_rn(__fmaf_rn(__fmaf_rn(-15.0f, q, a), 1.0f / 15.0f, q), __fadd_rn(mn[g], 0.0f));
    sz[g] = *reinterpret_cast<const uint32_t*>(&both);
  }
  if (!ok) return;
  uint8_t* codes = rec + (which ? I4_V_CODES : 0) + slot * I4_ROW;
  uint8_t* meta = rec + (which ? i4_v_meta(GK) : I4_META) + slot * i4_meta_row(GK);
  uint32_t w[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t mine = NG == 1 || c[u] < GK / 8 ? sz[0] : sz[NG - 1];
    const __half2 both = *reinterpret_cast<const __half2*>(&mine);
    w[u] = codes_of(x[u], __low2float(both), __high2float(both), wild);
    if (c[u] % (GK / 8) == 0) *reinterpret_cast<uint32_t*>(meta + 4 * (c[u] / (GK / 8))) = mine;
  }
  *reinterpret_cast<uint32_t*>(codes + 4 * c[0]) = w[0];
  *reinterpret_cast<uint32_t*>(codes + 4 * c[1]) = w[1];
}

// One warp takes 16 head rows (query, key and value heads in this order; in 4 bits key
// and value rows or query rows) of one token: four groups of 8 lanes, a lane holding both
// chunks of its channel pairs, so that the rotation needs no exchange and the cosines and sines are loaded
// once for all rows.  The kernel moves each byte once, and its traffic bounds it: in BF16
// all loads of a lane (8 x 16 B) are in flight together.
template <int GK, bool INTERLEAVED>
__global__ void __launch_bounds__(APP_THREADS, GK == 0 ? 1 : 7)
    paged_append_kernel(const __grid_constant__ PagedView p, const __grid_constant__ PagedRows rows,
                        const __grid_constant__ RopeArgs rope, const __grid_constant__ AppendRows in,
                        uint32_t kv_per_token, uint32_t per_token, uint32_t tasks) {
  const uint32_t task = (blockIdx.x * APP_THREADS + threadIdx.x) >> 5;
  if (task >= tasks) return;
  const int lane = threadIdx.x & 31, pc = lane & 7, sub = lane >> 3;
  const int hq = in.q ? in.Hq : 0;
  // a token's tasks: kv_per_token of key and value rows alone (4 bits), then those of query
  // rows (in BF16 with key and value rows behind them)
  const int row = static_cast<int>(task / per_token), of_token = static_cast<int>(task % per_token);
  const bool kv_only = GK != 0 && of_token < static_cast<int>(kv_per_token);
  const int head0 = (kv_only ? hq + of_token * APP_HEADS : (of_token - static_cast<int>(kv_per_token)) * APP_HEADS) + sub;
  const int total = GK == 0 || kv_only ? hq + 2 * p.Hkv : hq;

  // the lane's two chunks, and whether they hold rotated pairs; neighbours of a chunk are in
  // the next lane, so that an access of the warp takes whole sectors
  const int half_chunks = rope.table ? rope.dim / 16 : 0;   // half the rotated chunks
  int c[2];
  c[0] = INTERLEAVED || pc < half_chunks ? pc : pc + half_chunks;
  c[1] = INTERLEAVED || pc >= half_chunks ? pc + 8 : pc + half_chunks;
  const bool rot[2] = {c[0] < 2 * half_chunks, c[1] < 2 * half_chunks};   // (the same unless interleaved)
  auto load_row = [&](int r, uint32_t (&x)[2][4]) {
    const int h = head0 + 4 * r;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (h < total) {
      const uint16_t* src = h < hq           ? in.q + row * in.q_stride + h * D
                            : h < hq + p.Hkv ? in.k + row * in.k_stride + (h - hq) * D
                                             : in.v + row * in.v_stride + (h - hq - p.Hkv) * D;
      a = __ldcs(reinterpret_cast<const uint4*>(src + 8 * c[0]));
      b = __ldcs(reinterpret_cast<const uint4*>(src + 8 * c[1]));
    }
    x[0][0] = a.x, x[0][1] = a.y, x[0][2] = a.z, x[0][3] = a.w;
    x[1][0] = b.x, x[1][1] = b.y, x[1][2] = b.z, x[1][3] = b.w;
  };
  paged::grid_dep_launch();
  paged::grid_dep_wait();
  uint32_t x[APP_ROWS][2][4];
  load_row(0, x[0]);
  if (!kv_only) {
#pragma unroll
    for (int r = 1; r < APP_ROWS; ++r) load_row(r, x[r]);
  }
  const int i = find_req(rows, p.n, row);
  const int pos = rows.pos0[i] + (row - rows.row0[i]);
  // pair e of the lane: element e of both chunks, or elements 2e, 2e + 1 of the 16
  float cs[8], sn[8];
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (rot[u]) {
      const float* t = rope.table + (size_t)pos * rope.dim + (INTERLEAVED ? 4 * c[u] : 8 * pc + 4 * u);
      *reinterpret_cast<float4*>(cs + 4 * u) = *reinterpret_cast<const float4*>(t);
      *reinterpret_cast<float4*>(sn + 4 * u) = *reinterpret_cast<const float4*>(t + rope.dim / 2);
    }
  const bool writes_kv = total > hq && head0 + 4 * (APP_ROWS - 1) >= hq;
  const int64_t page = writes_kv ? page_of(p, i, pos) : -1;
  const int slot = pos % PAGE;
  auto rotate_row = [&](int h, uint32_t (&x)[2][4]) {
    if (h >= hq + p.Hkv) return;
    // (scalar operations: packed ones of two are contracted to fused multiply-adds)
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!rot[u]) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = bf_lo(x[u][k]), b = bf_hi(x[u][k]), co = cs[4 * u + k], si = sn[4 * u + k];
          x[u][k] = pack_bf(__fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si)),
                            __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si)));
        }
      }
    } else if (rot[0]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a0 = bf_lo(x[0][k]), a1 = bf_hi(x[0][k]), b0 = bf_lo(x[1][k]), b1 = bf_hi(x[1][k]);
        x[0][k] = pack_bf(__fsub_rn(__fmul_rn(a0, cs[2 * k]), __fmul_rn(b0, sn[2 * k])),
                          __fsub_rn(__fmul_rn(a1, cs[2 * k + 1]), __fmul_rn(b1, sn[2 * k + 1])));
        x[1][k] = pack_bf(__fadd_rn(__fmul_rn(b0, cs[2 * k]), __fmul_rn(a0, sn[2 * k])),
                          __fadd_rn(__fmul_rn(b1, cs[2 * k + 1]), __fmul_rn(a1, sn[2 * k + 1])));
      }
    }
  };
  if (!kv_only) {
#pragma unroll
    for (int r = 0; r < APP_ROWS; ++r) {
      const int h = head0 + 4 * r;
      rotate_row(h, x[r]);
      uint16_t* dst = nullptr;
      if (h < hq) {
        dst = in.q_out + ((size_t)row * in.Hq + h) * D;
      } else if (GK == 0 && h < total && page >= 0) {
        const int which = h >= hq + p.Hkv, kvh = h - hq - (which ? p.Hkv : 0);
        dst = static_cast<uint16_t*>(p.pool) + ((size_t)page * p.Hkv + kvh) * BF16_RECORD_ELEMS +
              (size_t)which * PAGE * D + (size_t)slot * D;
      }
      if (dst) {
        *reinterpret_cast<uint4*>(dst + 8 * c[0]) = make_uint4(x[r][0][0], x[r][0][1], x[r][0][2], x[r][0][3]);
        *reinterpret_cast<uint4*>(dst + 8 * c[1]) = make_uint4(x[r][1][0], x[r][1][1], x[r][1][2], x[r][1][3]);
      }
    }
  } else if constexpr (GK != 0) {
    // one copy of the quantiser's code (four do not fit the instruction cache: 102 us for
    // 16K tokens, 95 rolled up); the next row is loaded under it
#pragma unroll 1
    for (int r = 0; r < APP_ROWS; ++r) {
      const int h = head0 + 4 * r, which = h >= hq + p.Hkv, kvh = h - hq - (which ? p.Hkv : 0);
      uint32_t y[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[u][k] = x[0][u][k];
      if (r + 1 < APP_ROWS) load_row(r + 1, x[0]);
      rotate_row(h, y);
      // the whole warp takes part in the reductions' shuffles
      const bool ok = h < total && page >= 0;
      uint8_t* rec = static_cast<uint8_t*>(p.pool) + (ok ? ((size_t)page * p.Hkv + kvh) * i4_record(GK) : 0);
      if (__any_sync(0xffffffffu, ok)) store_int4<GK>(rec, which, slot, c, y, ok);
    }
  }
}

// ---- 4-bit read-back: one thread per word of 8 key codes and that of the values --
// Bound by its stores: K and V of 16K tokens of 8 heads as fp32 in 24.7 us (6.2 TB/s), as
// bf16 in 17.1 us (5.0 TB/s: half the bytes for the same loads and look-ups).
constexpr int READ_THREADS = 256;

// The 8 values s c + z of a word.  s c is exact in fp32 (11 + 4 bits), so a value is rounded
// once.  Pairs of codes become fp16 numbers 1024 + c (or 1024 + 16 c), then c.
template <bool F32>
__device__ __forceinline__ void put_values(void* out, size_t at, uint32_t w, float s, float z) {
  float y[8];
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {   // codes 2 half + odd and that + 4
      const uint32_t bits = ((w >> (8 * half)) & (odd ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
      __half2 c = *reinterpret_cast<const __half2*>(&bits);
      c = odd ? __hfma2(c, __half2half2(__ushort_as_half(0x2C00)), __half2half2(__ushort_as_half(0xD400)))   // / 16 - 64
              : __hadd2(c, __half2half2(__ushort_as_half(0xE400)));                                          // - 1024
      y[2 * half + odd] = fmaf(__low2float(c), s, z);
      y[2 * half + odd + 4] = fmaf(__high2float(c), s, z);
    }
  if constexpr (F32) {
    float* dst = static_cast<float*>(out) + at;
    if ((reinterpret_cast<uintptr_t>(out) & 31) == 0) {   // at once: stores of 16 bytes each send half of every sector
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(y[0]), "f"(y[1]),
                   "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7])
                   : "memory");
    } else {
      reinterpret_cast<float4*>(dst)[0] = make_float4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(y[4], y[5], y[6], y[7]);
    }
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
        make_uint4(pack_bf(y[0], y[1]), pack_bf(y[2], y[3]), pack_bf(y[4], y[5]), pack_bf(y[6], y[7]));
  }
}

template <int GK, bool F32>
__global__ void __launch_bounds__(READ_THREADS) int4_read_kernel(const __grid_constant__ PagedView p,
                                                                 const __grid_constant__ PagedRows rows, void* k_out,
                                                                 void* v_out, uint32_t heads) {
  // 16 threads a (row, head)
  const uint32_t rh = blockIdx.x * (READ_THREADS / 16) + threadIdx.x / 16, chunk = threadIdx.x & 15;
  if (rh >= heads) return;
  const int row = static_cast<int>(rh / static_cast<uint32_t>(p.Hkv)), head = static_cast<int>(rh - row * p.Hkv);
  const int i = find_req(rows, p.n, row);
  const int pos = rows.pos0[i] + (row - rows.row0[i]);
  paged::grid_dep_launch();
  paged::grid_dep_wait();
  const int64_t page = page_of(p, i, pos);
  uint32_t kw = 0, vw = 0;
  __half2 km = __half2half2(__ushort_as_half(0)), vm = km;
  if (page >= 0) {
    const uint8_t* rec = static_cast<const uint8_t*>(p.pool) + ((size_t)page * p.Hkv + head) * i4_record(GK);
    const int code = (pos % PAGE) * I4_ROW + 4 * chunk, meta = (pos % PAGE) * i4_meta_row(GK) + 4 * (chunk / (GK / 8));
    kw = *reinterpret_cast<const uint32_t*>(rec + code);
    vw = *reinterpret_cast<const uint32_t*>(rec + I4_V_CODES + code);
    km = *reinterpret_cast<const __half2*>(rec + I4_META + meta);
    vm = *reinterpret_cast<const __half2*>(rec + i4_v_meta(GK) + meta);
  }
  const size_t at = (size_t)rh * D + 8 * chunk;
  put_values<F32>(k_out, at, kw, __low2float(km), __high2float(km));
  put_values<F32>(v_out, at, vw, __low2float(vm), __high2float(vm));
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& p, const PagedRows& rows, const RopeArgs& rope, const AppendRows& in,
                                int gk, cudaStream_t s) {
  const int hq = in.q ? in.Hq : 0, tokens = rows.row0[p.n];
  auto tasks_for = [](int heads) { return (heads + APP_HEADS - 1) / APP_HEADS; };
  const uint32_t kv_per = gk == 0 ? 0 : tasks_for(2 * p.Hkv), per = kv_per + tasks_for(gk == 0 ? hq + 2 * p.Hkv : hq);
  const int64_t tasks = (int64_t)tokens * per;
  if (tasks * 32 > UINT32_MAX - APP_THREADS) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>((tasks * 32 + APP_THREADS - 1) / APP_THREADS);
  auto go = [&](auto kernel) {
    return paged::launch_dependent(kernel, grid, APP_THREADS, 0, s, p, rows, rope, in, kv_per, per,
                                   static_cast<uint32_t>(tasks));
  };
  if (gk == 0) return rope.interleaved ? go(paged_append_kernel<0, true>) : go(paged_append_kernel<0, false>);
  if (gk == 128) return rope.interleaved ? go(paged_append_kernel<128, true>) : go(paged_append_kernel<128, false>);
  return rope.interleaved ? go(paged_append_kernel<64, true>) : go(paged_append_kernel<64, false>);
}

cudaError_t launch_int4_read(const PagedView& p, const PagedRows& rows, int gk, void* k_out, void* v_out, bool f32,
                             cudaStream_t s) {
  const int64_t all = (int64_t)rows.row0[p.n] * p.Hkv;
  if (all > INT32_MAX) return cudaErrorInvalidValue;   // (1 TB of values)
  const uint32_t heads = static_cast<uint32_t>(all);
  const unsigned grid = (heads + READ_THREADS / 16 - 1) / (READ_THREADS / 16);
  auto go = [&](auto kernel) {
    return paged::launch_dependent(kernel, grid, READ_THREADS, 0, s, p, rows, k_out, v_out, heads);
  };
  if (gk == 128) return f32 ? go(int4_read_kernel<128, true>) : go(int4_read_kernel<128, false>);
  return f32 ? go(int4_read_kernel<64, true>) : go(int4_read_kernel<64, false>);
}

}  // namespace oscar
