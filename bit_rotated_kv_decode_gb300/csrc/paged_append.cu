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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "paged.h"

namespace oscar {
namespace {

constexpr int APP_THREADS = 128;
constexpr int APP_ROWS = 4;                    // head rows per lane group in flight
constexpr int APP_HEADS = 4 * APP_ROWS;        // head rows per warp: four groups of 8 lanes

struct alignas(16) Bf8 {
  uint16_t x[8];
};
__device__ __forceinline__ float bf_f(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t f_bf(float x) {
  const __nv_bfloat16 h = __float2bfloat16_rn(x);
  return *reinterpret_cast<const uint16_t*>(&h);
}

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
  const int32_t page = __ldg(p.table + (size_t)i * p.max_pages + pos / PAGE);
  if (page >= 0 && page < p.num_pages) return page;
  if (p.err) atomicOr(p.err, PAGED_ERR_PAGE);
  return -1;
}

// Quantise one head row held by 8 lanes, 16 channels each: chunks of 8 channels
// c[0] and c[1] with values x[0] and x[1].  Writes the codes and, from the lane
// that holds a group's first chunk, {s, z}.
template <int GK>
__device__ __forceinline__ void store_int4(uint8_t* rec, int which, int slot, const int (&c)[2], Bf8 (&x)[2], bool ok) {
  constexpr int NG = D / GK;
  float f[2][8], mn[NG], mx[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    mn[g] = INFINITY;
    mx[g] = -INFINITY;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float y = bf_f(x[u].x[e]);
      y = y == y ? fminf(fmaxf(y, -65504.0f), 65504.0f) : 0.0f;
      f[u][e] = y;
      lo = fminf(lo, y);
      hi = fmaxf(hi, y);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
      if (NG == 1 || c[u] / (GK / 8) == g) {
        mn[g] = fminf(mn[g], lo);
        mx[g] = fmaxf(mx[g], hi);
      }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
      mn[g] = fminf(mn[g], __shfl_xor_sync(0xffffffffu, mn[g], off));
      mx[g] = fmaxf(mx[g], __shfl_xor_sync(0xffffffffu, mx[g], off));
    }
  __half s[NG], z[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    z[g] = __float2half_rn(mn[g]);
    s[g] = __float2half_rn(__fdiv_rn(__fsub_rn(mx[g], mn[g]), 15.0f));
  }
  if (!ok) return;
  uint8_t* codes = rec + (which ? I4_V_CODES : 0) + slot * I4_ROW;
  uint8_t* meta = rec + (which ? i4_v_meta(GK) : I4_META) + slot * i4_meta_row(GK);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int g = NG == 1 ? 0 : c[u] / (GK / 8);
    const __half sh = NG == 1 || g == 0 ? s[0] : s[NG - 1], zh = NG == 1 || g == 0 ? z[0] : z[NG - 1];
    const float sf = __half2float(sh), zf = __half2float(zh);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = rintf(__fdiv_rn(__fsub_rn(f[u][e], zf), sf));
      const int code = sf == 0.0f ? 0 : static_cast<int>(fminf(fmaxf(t, 0.0f), 15.0f));
      w |= static_cast<uint32_t>(code) << (4 * e);
    }
    *reinterpret_cast<uint32_t*>(codes + 4 * c[u]) = w;
    if (c[u] % (GK / 8) == 0)
      *reinterpret_cast<uint32_t*>(meta + 4 * g) =
          static_cast<uint32_t>(__half_as_ushort(sh)) | (static_cast<uint32_t>(__half_as_ushort(zh)) << 16);
  }
}

// One warp takes 16 head rows (query, key and value heads in this order) of one
// token: four groups of 8 lanes, a lane holding both chunks of its channel pairs,
// so that the rotation needs no exchange and the cosines and sines are loaded
// once for all rows.  The kernel moves each byte once; all loads of a lane
// (8 x 16 B) are in flight together.
template <int GK>
__global__ void __launch_bounds__(APP_THREADS) paged_append_kernel(const __grid_constant__ PagedView p,
                                                                   const __grid_constant__ PagedRows rows,
                                                                   const __grid_constant__ RopeArgs rope,
                                                                   const __grid_constant__ AppendRows in,
                                                                   int tasks_per_token, int64_t tasks) {
  const int64_t task = ((int64_t)blockIdx.x * APP_THREADS + threadIdx.x) >> 5;
  if (task >= tasks) return;
  const int lane = threadIdx.x & 31, pc = lane & 7, sub = lane >> 3;
  const int row = static_cast<int>(task / tasks_per_token);
  const int head0 = static_cast<int>(task % tasks_per_token) * APP_HEADS + sub;
  const int i = find_req(rows, p.n, row);
  const int pos = rows.pos0[i] + (row - rows.row0[i]);
  const int hq = in.q ? in.Hq : 0, total = hq + 2 * p.Hkv;

  // the lane's two chunks, and whether they hold rotated pairs
  int c[2];
  const int half_chunks = rope.dim / 16;   // rotated pairs of chunks (half layout)
  bool rot = rope.table != nullptr;
  if (rope.interleaved) {
    c[0] = 2 * pc;
    c[1] = 2 * pc + 1;
    rot = rot && pc < half_chunks;
  } else if (rot && pc < half_chunks) {
    c[0] = pc;
    c[1] = pc + half_chunks;
  } else {
    rot = false;
    c[0] = rope.table ? 2 * pc : 2 * pc;
    c[1] = c[0] + 1;
  }
  Bf8 x[APP_ROWS][2];
#pragma unroll
  for (int r = 0; r < APP_ROWS; ++r) {
    const int h = head0 + 4 * r;
    if (h >= total) continue;
    const uint16_t* src = h < hq            ? in.q + row * in.q_stride + (int64_t)h * D
                          : h < hq + p.Hkv  ? in.k + row * in.k_stride + (int64_t)(h - hq) * D
                                            : in.v + row * in.v_stride + (int64_t)(h - hq - p.Hkv) * D;
    x[r][0] = *reinterpret_cast<const Bf8*>(src + 8 * c[0]);
    x[r][1] = *reinterpret_cast<const Bf8*>(src + 8 * c[1]);
  }
  // pair e of the lane: channels (c[0], c[1]) element e, or (2e, 2e + 1) of the two chunks
  float cs[8], sn[8];
  if (rot) {
    const float* t = rope.table + (size_t)pos * rope.dim + 8 * pc;
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      *reinterpret_cast<float4*>(cs + e) = __ldg(reinterpret_cast<const float4*>(t + e));
      *reinterpret_cast<float4*>(sn + e) = __ldg(reinterpret_cast<const float4*>(t + rope.dim / 2 + e));
    }
  }
  const bool writes_kv = head0 + 4 * (APP_ROWS - 1) >= hq;
  const int64_t page = writes_kv ? page_of(p, i, pos) : -1;
  const int slot = pos % PAGE;
#pragma unroll
  for (int r = 0; r < APP_ROWS; ++r) {
    const int h = head0 + 4 * r;
    if (rot && h < hq + p.Hkv) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint16_t& xa = rope.interleaved ? x[r][e >> 2].x[2 * (e & 3)] : x[r][0].x[e];
        uint16_t& xb = rope.interleaved ? x[r][e >> 2].x[2 * (e & 3) + 1] : x[r][1].x[e];
        const float a = bf_f(xa), b = bf_f(xb);
        xa = f_bf(__fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e])));
        xb = f_bf(__fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e])));
      }
    }
    const bool is_q = h < hq;
    const int which = h >= hq + p.Hkv, kvh = h - hq - (which ? p.Hkv : 0);
    if (is_q) {
      uint16_t* dst = in.q_out + ((size_t)row * in.Hq + h) * D;
      *reinterpret_cast<Bf8*>(dst + 8 * c[0]) = x[r][0];
      *reinterpret_cast<Bf8*>(dst + 8 * c[1]) = x[r][1];
    }
    const bool ok = !is_q && h < total && page >= 0;
    if constexpr (GK == 0) {
      if (ok) {
        uint16_t* dst = static_cast<uint16_t*>(p.pool) + ((size_t)page * p.Hkv + kvh) * BF16_RECORD_ELEMS +
                        (size_t)which * PAGE * D + (size_t)slot * D;
        *reinterpret_cast<Bf8*>(dst + 8 * c[0]) = x[r][0];
        *reinterpret_cast<Bf8*>(dst + 8 * c[1]) = x[r][1];
      }
    } else {
      // the whole warp takes part in the reductions' shuffles
      uint8_t* rec = static_cast<uint8_t*>(p.pool) + (ok ? ((size_t)page * p.Hkv + kvh) * i4_record(GK) : 0);
      if (__any_sync(0xffffffffu, ok)) store_int4<GK>(rec, which, slot, c, x[r], ok);
    }
  }
}

// ---- 4-bit read-back: one thread per word of 8 codes -------------------------
constexpr int READ_THREADS = 256;

template <int GK, bool F32>
__global__ void __launch_bounds__(READ_THREADS) int4_read_kernel(const __grid_constant__ PagedView p,
                                                                 const __grid_constant__ PagedRows rows, void* k_out,
                                                                 void* v_out, int64_t words) {
  const int64_t idx = (int64_t)blockIdx.x * READ_THREADS + threadIdx.x;
  if (idx >= words) return;
  // word = ((row Hkv + head) 2 + which) 16 + chunk
  const int chunk = static_cast<int>(idx & 15), which = static_cast<int>((idx >> 4) & 1);
  const int64_t rh = idx >> 5;
  const int row = static_cast<int>(rh / p.Hkv), head = static_cast<int>(rh % p.Hkv);
  const int i = find_req(rows, p.n, row);
  const int pos = rows.pos0[i] + (row - rows.row0[i]);
  const int64_t page = page_of(p, i, pos);
  uint32_t w = 0;
  float s = 0.0f, z = 0.0f;
  if (page >= 0) {
    const uint8_t* rec = static_cast<const uint8_t*>(p.pool) + ((size_t)page * p.Hkv + head) * i4_record(GK);
    const int slot = pos % PAGE;
    w = *reinterpret_cast<const uint32_t*>(rec + (which ? I4_V_CODES : 0) + slot * I4_ROW + 4 * chunk);
    const __half2 m = *reinterpret_cast<const __half2*>(rec + (which ? i4_v_meta(GK) : I4_META) +
                                                        slot * i4_meta_row(GK) + 4 * (chunk / (GK / 8)));
    s = __low2float(m);
    z = __high2float(m);
  }
  // s code is exact in fp32 (11 + 4 bits), so the value is rounded once
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(static_cast<float>((w >> (4 * e)) & 15), s, z);
  const size_t at = (size_t)rh * D + 8 * chunk;
  if constexpr (F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(which ? v_out : k_out) + at);
    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    Bf8 b;
#pragma unroll
    for (int e = 0; e < 8; ++e) b.x[e] = f_bf(y[e]);
    *reinterpret_cast<Bf8*>(static_cast<uint16_t*>(which ? v_out : k_out) + at) = b;
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& p, const PagedRows& rows, const RopeArgs& rope, const AppendRows& in,
                                int gk, cudaStream_t s) {
  const int heads = (in.q ? in.Hq : 0) + 2 * p.Hkv;
  const int per_token = (heads + APP_HEADS - 1) / APP_HEADS;
  const int64_t tasks = (int64_t)rows.row0[p.n] * per_token;
  const int64_t blocks = (tasks * 32 + APP_THREADS - 1) / APP_THREADS;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (gk == 0)
    paged_append_kernel<0><<<grid, APP_THREADS, 0, s>>>(p, rows, rope, in, per_token, tasks);
  else if (gk == 128)
    paged_append_kernel<128><<<grid, APP_THREADS, 0, s>>>(p, rows, rope, in, per_token, tasks);
  else
    paged_append_kernel<64><<<grid, APP_THREADS, 0, s>>>(p, rows, rope, in, per_token, tasks);
  return cudaGetLastError();
}

cudaError_t launch_int4_read(const PagedView& p, const PagedRows& rows, int gk, void* k_out, void* v_out, bool f32,
                             cudaStream_t s) {
  const int64_t words = (int64_t)rows.row0[p.n] * p.Hkv * 32;
  const int64_t blocks = (words + READ_THREADS - 1) / READ_THREADS;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (gk == 128) {
    if (f32) int4_read_kernel<128, true><<<grid, READ_THREADS, 0, s>>>(p, rows, k_out, v_out, words);
    else int4_read_kernel<128, false><<<grid, READ_THREADS, 0, s>>>(p, rows, k_out, v_out, words);
  } else {
    if (f32) int4_read_kernel<64, true><<<grid, READ_THREADS, 0, s>>>(p, rows, k_out, v_out, words);
    else int4_read_kernel<64, false><<<grid, READ_THREADS, 0, s>>>(p, rows, k_out, v_out, words);
  }
  return cudaGetLastError();
}

}  // namespace oscar
