// Tokens of the three-segment cache as values in their own basis: BF16 tokens as they are,
// history tokens x = (z + s c) R^T (codes, scale and zero: "TogetherAI开源OSCAR" (ModelScope),
// section "OSCAR的设计"; the rotation undone as "Together AI Open-Sources OSCAR" (MarkTechPost),
// section "What OSCAR Does Differently", defines it).
//
// read_history_kernel takes 128 history tokens of one kv head, K or V, at a time, whatever
// requests they are of: a product of 128 x 128 x 128 on tcgen05.
//   bf16 outputs  the values z + s c in fp16, times a power of two of the token's that keeps them in
//                 range, by R in fp16: each off by 2^-11, an eighth of what the output's rounding adds;
//   fp32 outputs  with c' = c - 1, whole numbers that any type holds,
//                   x_j = s (c' R^T)_j + (z + s) sum_i R_ji     (per group of channels),
//                 R in three bf16 parts (24 bits), the small ones first, the sums of its rows
//                 once per CTA; two groups of channels have an accumulator each.
//
// Bound by the stores (30K tokens of 8 kv heads: bf16 32 us, 123 MB written of 141 moved; fp32 63 us, 246 of 264:
// 4.2 to 4.4 TB/s) and 8 us of set-up.
//
// Two to four groups of four warps per CTA take tiles in turn: what one waits for (its codes, two
// loads apart, and its products), the others' outputs cover.
// A lane of the accumulator is an output channel for fp32 outputs (R times the tokens), so that a
// warp stores 128 neighbouring bytes straight from the registers that it reads; for bf16 it is a token,
// whose row goes through shared memory, eight lanes a piece of 128 bytes (30K tokens: fp32 63 us, 73
// that way; bf16 67 us the first way, its stores being half as wide).
#include <atomic>
#include <type_traits>

#include "append_device.cuh"
#include "chunk.h"
#include "values_device.cuh"

namespace oscar {
namespace {

using namespace paged;

constexpr int RD_ROWS = 128;

// Groups that shared memory and the 512 columns of Tensor Memory hold.
__host__ __device__ constexpr int read_groups(int gk, bool f32) { return !f32 ? 4 : gk == 64 ? 2 : 3; }

template <int GK, bool F32>
struct alignas(1024) ReadSmem {
  static constexpr int PARTS = F32 ? 3 : 1, GROUPS = read_groups(GK, F32);
  alignas(1024) uint8_t r[PARTS][TILE_BYTES];           // R, smallest part first: two halves of 64 inputs, [128 outputs][128 B] swizzled
  alignas(1024) uint8_t code[GROUPS][TILE_BYTES];       // values or c' of a tile, likewise
  // fp32: sums of R's rows over a group of channels; of a tile's tokens and those of the next s and z + s of each
  // group of channels, and rows of the output (-1: none).  bf16: per warp 128 bytes of its 32 rows
  struct Fp32 {
    alignas(16) float sum[2][D];
    alignas(16) float2 step[GROUPS][2][D / GK][RD_ROWS];
    alignas(16) int32_t to[GROUPS][2][RD_ROWS];
  };
  struct Bf16 {
    alignas(16) uint8_t out[GROUPS * 4][32 * 128];
  };
  std::conditional_t<F32, Fp32, Bf16> x;
  uint64_t done[GROUPS];
  uint32_t tmem;
};
static_assert(sizeof(ReadSmem<128, true>) + 1024 <= 232448 && sizeof(ReadSmem<128, false>) + 1024 <= 232448,
              "shared memory of a CTA");

__device__ __forceinline__ uint32_t tile_at(int row, int part) {
  return (part >> 3) * (TILE_BYTES / 2) + row * 128 + (((part & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(RD_ROWS) : "memory");
}
__device__ __forceinline__ bool group_all(int group, bool mine) {
  int all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.b32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(static_cast<int>(mine)), "r"(group + 1), "n"(RD_ROWS)
      : "memory");
  return all != 0;
}

// The 16 codes of a word as c - 1: bf16x2 i holds channels i and i + 8.  A code in the low mantissa bits of 2^e,
// e such that they count ones, is 2^e + c.
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i % 3, shift = 2 * (i - at);   // three codes fit the mantissa without a shift
    const uint32_t base = 0x4300u - (2u * at << 7), less = base | (1u << (2 * at));   // 2^(7 - 2 at), and one more
    const uint32_t bits = ((w >> shift) & (0x00030003u << (2 * at))) | (base | base << 16);
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&bits),
                                     __halves2bfloat162(__ushort_as_bfloat16(less), __ushort_as_bfloat16(less)));
    x[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <int GK, bool F32>
__global__ void __launch_bounds__(read_groups(GK, F32) * RD_ROWS, 1)
    read_history_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ReadArgs A, int tiles,
                        int per_matrix) {
  extern __shared__ uint8_t rd_raw[];
  using Smem = ReadSmem<GK, F32>;
  Smem& sm = *reinterpret_cast<Smem*>(rd_raw + (-smem_u32(rd_raw) & 1023u));
  constexpr int NG = D / GK, PARTS = Smem::PARTS, GROUPS = Smem::GROUPS, THREADS = GROUPS * RD_ROWS;
  constexpr int SUMS = F32 ? NG : 1;             // accumulators of a tile
  constexpr uint32_t IDESC = F32 ? IDESC_QK : IDESC_QK_F16;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int group = warp >> 2, r = threadIdx.x & (RD_ROWS - 1);
  const int matrix = blockIdx.x / per_matrix, part = blockIdx.x % per_matrix;
  const int head = matrix >> 1, which = matrix & 1;
  const float* R = (which ? c.rot_v : c.rot_k) + ((size_t)A.layer * c.Hkv + head) * D * D;

  if (threadIdx.x == 0) {
    for (int g = 0; g < GROUPS; ++g) mbar_init(&sm.done[g], 1);
    mbar_init_fence();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // R, written once at the cache's creation (before the grid's dependency): 16 inputs at a time, in the order
  // that unpack_*() leave channels in
#pragma unroll 2
  for (int i = threadIdx.x; i < D * (D / 16); i += THREADS) {
    const int n = i / (D / 16), p = i % (D / 16);
    float f[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(f + 4 * j) = reinterpret_cast<const float4*>(R + (size_t)n * D + 16 * p)[j];
#pragma unroll
    for (int u = PARTS - 1; u >= 0; --u) {
      uint32_t x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (F32) {
          x[j] = bf16x2(f[j], f[j + 8]);
          f[j] -= __uint_as_float(x[j] << 16);
          f[j + 8] -= __uint_as_float(x[j] & 0xffff0000u);
        } else {
          x[j] = f16x2(f[j], f[j + 8]);
        }
      }
      *reinterpret_cast<uint4*>(sm.r[u] + tile_at(n, 2 * p)) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(sm.r[u] + tile_at(n, 2 * p + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
  if constexpr (F32) {   // sums of R's rows: thread (output, half of the inputs)
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
      const int n = i & (D - 1), h = i >> 7;
      float s = 0.0f;
#pragma unroll 8
      for (int j = 0; j < D / 2; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(R + (size_t)n * D + h * (D / 2) + j);
        s += (f.x + f.y) + (f.z + f.w);
      }
      sm.x.sum[h][n] = s;
    }
  }
  fence_async_smem();
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (F32 && NG == 1) {
    if (threadIdx.x < D) sm.x.sum[0][threadIdx.x] += sm.x.sum[1][threadIdx.x];
    __syncthreads();
  }

  const int total = A.hist[A.n];
  // (few tiles go to CTAs of their own)
  const int step = GROUPS * per_matrix, first = part + per_matrix * group;
  uint4 words[2];          // codes of this thread's row of the next tile
  uint32_t meta[NG];       // its {s, z}
  int to = -1;             // its row of the output
  int scale = 0;           // exponent of the staged token's values
  auto fetch = [&](int t) {
    const int i = t * RD_ROWS + r;
    to = -1;
    words[0] = words[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < NG; ++n) meta[n] = 0;
    if (i >= total) return;
    int ri = 0, hi = A.n;
    while (hi - ri > 1) {
      const int mid = (ri + hi) >> 1;
      if (A.hist[mid] <= i) ri = mid; else hi = mid;
    }
    const int off = i - A.hist[ri], at = A.first[ri] + off - SINK, row = at % PAGE;
    to = A.out0[ri] + off;
    const int page = c.hist_pt[(size_t)A.slot[ri] * c.max_pages + at / PAGE];
    if (page < 0 || page >= c.n_int2_pages) {
      atomicOr(c.err, ERR_INT2_PAGE);
      return;   // (zeros)
    }
    const uint8_t* rec = int2_record(c, A.layer, page, head);
    const uint4* code = reinterpret_cast<const uint4*>(rec + (which ? V_CODES_OFF : K_CODES_OFF) + row * CODE_BYTES);
    words[0] = code[0];
    words[1] = code[1];
    const uint32_t* m = reinterpret_cast<const uint32_t*>(rec + (which ? v_meta_off_for(GK) : k_meta_off_for(GK)) +
                                                         row * meta_bytes_for(GK));
#pragma unroll
    for (int n = 0; n < NG; ++n) meta[n] = m[n];
  };
  // the fetched token into the group's tile, the buf-th of its two
  auto stage = [&](int buf) {
    if constexpr (F32) {
      sm.x.to[group][buf][r] = to;
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const float s = __half2float(__ushort_as_half(meta[n] & 0xffff)), z = __half2float(__ushort_as_half(meta[n] >> 16));
        sm.x.step[group][buf][n][r] = make_float2(s, z + s);
      }
    }
    const uint32_t w[8] = {words[0].x, words[0].y, words[0].z, words[0].w, words[1].x, words[1].y, words[1].z, words[1].w};
    __half2 s[5], z;
    float down = 0.0f;
    if constexpr (!F32) {
      scale = value_exponent(largest_value(meta));
      down = pow2(-scale);
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t x[8];
      if constexpr (F32) {
        unpack_codes(w[p], x);
      } else {
        if (p % (8 / NG) == 0) value_steps(meta[p / (8 / NG)], down, s, z);
        unpack_values(w[p], s, z, x);
      }
      *reinterpret_cast<uint4*>(sm.code[group] + tile_at(r, 2 * p)) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4*>(sm.code[group] + tile_at(r, 2 * p + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
    }
    fence_async_smem();
  };
  const uint32_t acc0 = 128 * SUMS * group;
  auto multiply = [&]() {
    if ((warp & 3) != 0) return;
    tc_fence_after();
    const uint64_t a = desc_kmajor(smem_u32(sm.code[group]));
#pragma unroll
    for (int n = 0; n < SUMS; ++n)
#pragma unroll
      for (int u = 0; u < PARTS; ++u) {
        const uint64_t b = desc_kmajor(smem_u32(sm.r[u]));
#pragma unroll
        for (int s = 8 / SUMS * n; s < 8 / SUMS * (n + 1); ++s) {
          const uint64_t off = ((s >> 2) * (TILE_BYTES / 2) + (s & 3) * 32) >> 4;
          mma_ss(acc0 + 128 * n, (F32 ? b : a) + off, (F32 ? a : b) + off, IDESC, u > 0 || s > 8 / SUMS * n);
        }
      }
    mma_commit(&sm.done[group]);
  };

  bool ok = true;
  int count = 0, now = -1;
  if (first < tiles) {
    fetch(first);
    stage(0);
    now = to;
    tc_fence_before();
    group_sync(group);
    multiply();
    if (first + step < tiles) fetch(first + step);
  }
  constexpr int SIZE = F32 ? 4 : 2;
  char* const out = static_cast<char*>(which ? A.v_out : A.k_out) + (size_t)head * (D * SIZE);
  const size_t row_bytes = (size_t)c.Hkv * (D * SIZE);
  const uint32_t acc = (static_cast<uint32_t>(32 * (warp & 3)) << 16) + acc0;
  for (int t = first; t < tiles && ok; t += step, ++count) {
    const int buf = count & 1, mine = now;   // (this thread's token, staged a tile ago: its row and exponent)
    const float up = pow2(scale);
    const bool more = t + step < tiles;
    ok = group_all(group, mbar_wait(&sm.done[group], count & 1));
    if (!ok) break;
    tc_fence_after();
    if (more) {   // the next tile, fetched while the last one went out; the one after it is on its way meanwhile
      stage(buf ^ 1);
      now = to;
      if (t + 2 * step < tiles) fetch(t + 2 * step);
    }
    if constexpr (F32) {
      const int ch = 32 * (warp & 3) + lane;   // this thread's output channel
      const float sum0 = sm.x.sum[0][ch], sum1 = NG == 2 ? sm.x.sum[1][ch] : 0.0f;
#pragma unroll 1
      for (int col = 0; col < RD_ROWS; col += 32) {   // 32 tokens
        uint32_t d[SUMS][32];
#pragma unroll
        for (int n = 0; n < SUMS; ++n) tmem_ld32(acc + 128 * n + col, d[n]);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const int4 to4 = *reinterpret_cast<const int4*>(&sm.x.to[group][buf][col + i]);
          const int rows[4] = {to4.x, to4.y, to4.z, to4.w};
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const float4 u = *reinterpret_cast<const float4*>(&sm.x.step[group][buf][0][col + i + j]);
            float y0 = fmaf(u.x, __uint_as_float(d[0][i + j]), u.y * sum0), y1 = fmaf(u.z, __uint_as_float(d[0][i + j + 1]), u.w * sum0);
            if constexpr (NG == 2) {
              const float4 v = *reinterpret_cast<const float4*>(&sm.x.step[group][buf][NG - 1][col + i + j]);
              y0 += fmaf(v.x, __uint_as_float(d[SUMS - 1][i + j]), v.y * sum1);
              y1 += fmaf(v.z, __uint_as_float(d[SUMS - 1][i + j + 1]), v.w * sum1);
            }
            if (rows[j] >= 0) reinterpret_cast<float*>(out + rows[j] * row_bytes)[ch] = y0;
            if (rows[j + 1] >= 0) reinterpret_cast<float*>(out + rows[j + 1] * row_bytes)[ch] = y1;
          }
        }
      }
    } else {
      uint8_t* turn = sm.x.out[warp];
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {   // 64 channels
        uint32_t w[32];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t d[32];
          tmem_ld32(acc + 64 * half + 32 * k, d);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            w[16 * k + j] = bf16x2(__uint_as_float(d[2 * j]) * up, __uint_as_float(d[2 * j + 1]) * up);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(turn + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rw = 4 * k + lane / 8, row = __shfl_sync(0xffffffffu, mine, rw);
          const uint4 v = *reinterpret_cast<const uint4*>(turn + rw * 128 + (((lane & 7) ^ (rw & 7)) << 4));
          if (row >= 0) *reinterpret_cast<uint4*>(out + row * row_bytes + 128 * half + 16 * (lane & 7)) = v;
        }
        __syncwarp();
      }
    }
    if (more) {
      tc_fence_before();
      group_sync(group);
      multiply();
    }
  }
  if (!ok && lane == 0) atomicOr(c.err, ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(0u) : "memory");
  }
}

// Tokens that the sink or the recent window holds: 16 lanes a row of one kv head, K or V.
constexpr int RB_THREADS = 256;
template <bool F32>
__global__ void __launch_bounds__(RB_THREADS)
    read_bf16_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ReadArgs A) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t unit = ((int64_t)blockIdx.x * RB_THREADS + threadIdx.x) / (D / 8);   // (row, kv head, K or V)
  const int part = threadIdx.x % (D / 8), which = static_cast<int>(unit & 1);
  const int head = static_cast<int>((unit >> 1) % c.Hkv);
  const int64_t i = (unit >> 1) / c.Hkv;
  if (i >= A.near[A.n]) return;
  int ri = 0, hi = A.n;
  while (hi - ri > 1) {
    const int mid = (ri + hi) >> 1;
    if (A.near[mid] <= i) ri = mid; else hi = mid;
  }
  // the request's tokens that are no history: those before it, then those after
  const int at = static_cast<int>(i) - A.near[ri], hist = A.hist[ri + 1] - A.hist[ri];
  const int before = A.first[ri] - A.start[ri], off = at < before ? at : at + hist, pos = A.start[ri] + off;
  const int page = c.bf16_pt[(size_t)A.slot[ri] * BF16_PAGES_PER_REQ + (pos < SINK ? 0 : 1 + (pos - SINK) % RECENT / PAGE)];
  uint4 v = make_uint4(0, 0, 0, 0);
  if (page < 0 || page >= c.n_bf16_pages) {
    if (part == 0) atomicOr(c.err, ERR_BF16_PAGE);
  } else {
    v = reinterpret_cast<const uint4*>(bf16_row(c, A.layer, page, head, which, pos % PAGE))[part];
  }
  const size_t row = (size_t)(A.out0[ri] - before + off) * c.Hkv + head;
  char* out = static_cast<char*>(which ? A.v_out : A.k_out) + row * (D * (F32 ? 4 : 2));
  if constexpr (F32) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 2; ++j)
      reinterpret_cast<uint4*>(out)[2 * part + j] =
          make_uint4(w[2 * j] << 16, w[2 * j] & 0xffff0000u, w[2 * j + 1] << 16, w[2 * j + 1] & 0xffff0000u);
  } else {
    reinterpret_cast<uint4*>(out)[part] = v;
  }
}

template <int GK, bool F32>
cudaError_t launch_history(const DevCache& c, const ReadArgs& a, int sms, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(ReadSmem<GK, F32>)) + 1024;
  static std::atomic<unsigned> done;   // devices that have been set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(done.load() & (1u << dev))) {
    e = cudaFuncSetAttribute(read_history_kernel<GK, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 32) done.fetch_or(1u << dev);
  }
  // CTAs for each of the 2 Hkv matrices: one per SM in all, none without a tile
  const int tiles = (a.hist[a.n] + RD_ROWS - 1) / RD_ROWS, matrices = 2 * c.Hkv;
  const int fair = sms / matrices > 1 ? sms / matrices : 1, per_matrix = tiles < fair ? tiles : fair;
  return launch_dependent(read_history_kernel<GK, F32>, static_cast<unsigned>(matrices * per_matrix), read_groups(GK, F32) * RD_ROWS, bytes,
                          s, c, a, tiles, per_matrix);
}

}  // namespace

cudaError_t launch_read_history(const DevCache& c, const ReadArgs& a, bool f32, int sms, cudaStream_t s) {
  if (c.gk == 64) return f32 ? launch_history<64, true>(c, a, sms, s) : launch_history<64, false>(c, a, sms, s);
  return f32 ? launch_history<128, true>(c, a, sms, s) : launch_history<128, false>(c, a, sms, s);
}

cudaError_t launch_read_bf16(const DevCache& c, const ReadArgs& a, bool f32, cudaStream_t s) {
  const int64_t threads = (int64_t)a.near[a.n] * c.Hkv * 2 * (D / 8);
  return launch_dependent(f32 ? read_bf16_kernel<true> : read_bf16_kernel<false>,
                          static_cast<unsigned>((threads + RB_THREADS - 1) / RB_THREADS), RB_THREADS, 0, s, c, a);
}

}  // namespace oscar
