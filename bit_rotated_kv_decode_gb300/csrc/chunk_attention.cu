// Attention of a chunk of new tokens of each request over the three-segment cache and, causally,
// over the chunk itself ("TogetherAI开源OSCAR" (ModelScope), section "OSCAR的设计": unpack, scale and
// zero, online-softmax merge of the segments; "Together AI Open-Sources OSCAR" (MarkTechPost),
// section "The Serving System").  Four kernels:
//   rotate_queries_kernel  q R_K in fp16, each row scaled by a power of two, its channels in the
//                          order that unpacking leaves the codes in;
//   chunk_scan_kernel      the history: partial rows (unnormalised sums, maximum, sum);
//   paged_prefill_kernel   the BF16 tokens and the new ones, likewise (paged_prefill_device.cuh);
//   chunk_merge_kernel     their sum, the history's times R_V^T, over the weights' sum.
//
// chunk_scan_kernel: a CTA takes 128 keys at a time.  Four warps unpack them, a key a thread,
// into fp16 values (z + s c) / 2 in shared memory (the half keeps thresholds up to 65504 in
// range; rounded once, half a step 2^-12), from codes that were fetched into registers a step
// before.  Per key tile and chain
//   S = Q K^T            128 x 128 x 128, tcgen05.mma, both operands in shared memory
//   p = exp2(S scale - m + 11)   one thread per row; fp16 (2^-12; the shift keeps weights down to
//                        2^-25 of the row's largest in full, where fp16 alone would flush them)
//   O = O + P V          tcgen05.mma, P from TMEM, O in TMEM
// The two chains are two tiles of 128 query rows (a row being a (token, head of the group) pair)
// that share every key, or, where a kv head has 128 rows or fewer, every other key tile each of
// the one tile of queries: a chain by itself is S, softmax, PV one after another.
//
// Bytes of history are few (72 a token-head): with 20 rows the scan is bound by unpacking into
// shared memory and reading it back, with 256 by the tensor core.  Work is a line of key tiles,
// segment by segment -- (request, kv head, 256 rows) -- with some set-up units in front of each,
// cut into one equal range per SM: a long request is spread over all of them, and none waits for
// the last segment.
#include <atomic>

#include "append_device.cuh"
#include "chunk.h"
#include "tcgen05_device.cuh"

namespace oscar {
namespace {

using namespace paged;

constexpr int SC_THREADS = 512;                // softmax of chain 0, of chain 1, unpacking, the others
constexpr int SC_UNPACK_WARP = 8, SC_MMA_WARP = 12, SC_LOAD_WARP = 14;
// Registers a thread: 128 at launch, then 168 for the softmax's two warpgroups, 104 for the one
// that unpacks, 72 for the last.
constexpr int SC_REGS = 128, SC_SOFTMAX_REGS = 168, SC_UNPACK_REGS = 104, SC_OTHER_REGS = 72;
static_assert(2 * SC_SOFTMAX_REGS + SC_UNPACK_REGS + SC_OTHER_REGS <= 4 * SC_REGS,
              "a split above the launch's registers waits forever");
constexpr int SC_STAGES = 2;                   // of V of a key tile and K of the next
constexpr int SC_ROWS = 128, SC_KEYS = 128;
constexpr int SC_FIRST = 64;                   // keys of P handed over first
constexpr float SC_LAZY = 4.0f;                // the softmax reference moves only when exceeded by 2^4
constexpr float SC_SHIFT = 11.0f;              // weights are at most 2^15, and fp16's steps below 2^-14 cost nothing

struct alignas(1024) ScanSmem {
  alignas(1024) uint8_t q[2][TILE_BYTES];                // two halves of 64 channels, [128 rows][128 B] swizzled
  alignas(1024) uint8_t kv[SC_STAGES][2][TILE_BYTES];    // V of an earlier key tile, K of this one
  alignas(16) uint8_t out[8][32 * 128];                  // per softmax warp: 128 bytes of its 32 rows
  uint64_t q_full, q_empty, kv_full[SC_STAGES], kv_empty[SC_STAGES];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_empty[2], turn[2];
  uint32_t tmem;
};
static_assert(sizeof(ScanSmem) + 1024 <= 232448, "shared memory of a CTA");

__device__ __forceinline__ uint32_t tile_at(int row, int part) {
  return (part >> 3) * (TILE_BYTES / 2) + row * 128 + (((part & 7) ^ (row & 7)) << 4);
}

// A CTA's walk along its range of the line of key tiles.
struct Segment {
  int req, head, block;    // request of the launch, kv head, block of rows
  int j0, j1;              // key tiles
  int64_t start, index;    // first unit on the line; segment number
};
struct Walk {
  int64_t lo, hi;          // the CTA's units that are left
  Segment s;
  __device__ static Walk begin(const ScanArgs& A) {
    Walk w;
    w.lo = chunk_cut(A, blockIdx.x);
    w.hi = chunk_cut(A, blockIdx.x + 1);
    int a = 0, b = A.n;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (A.cost[mid] <= w.lo) a = mid; else b = mid;
    }
    const int64_t each = A.tiles[a] + A.setup, k = (w.lo - A.cost[a]) / each;
    w.s.req = a;
    w.s.head = static_cast<int>(k / A.blocks[a]);
    w.s.block = static_cast<int>(k % A.blocks[a]);
    w.s.start = A.cost[a] + k * each;
    w.s.index = A.segment[a] + k;
    return w;
  }
  // the next segment of which the range has key tiles; false at its end
  __device__ bool next(const ScanArgs& A) {
    while (lo < hi) {
      const int64_t first = s.start + A.setup, end = first + A.tiles[s.req];
      if (lo < end) {
        s.j0 = static_cast<int>((lo > first ? lo : first) - first);
        s.j1 = static_cast<int>((hi < end ? hi : end) - first);
        if (s.j0 < s.j1) return true;
        return false;   // only set-up units are left
      }
      step(A);
    }
    return false;
  }
  __device__ void done(const ScanArgs& A) {   // the segment that next() gave is behind
    lo = s.start + A.setup + s.j1;
    if (s.j1 == A.tiles[s.req]) step(A);
  }
  __device__ void step(const ScanArgs& A) {
    s.start += A.tiles[s.req] + A.setup;
    ++s.index;
    if (++s.block == A.blocks[s.req]) {
      s.block = 0;
      if (++s.head == A.Hkv) {
        s.head = 0;
        ++s.req;
      }
    }
    if (lo < s.start) lo = s.start;
  }
};

// The 16 codes of a word as (z + s c) / 2, s and z given as halves in both halves: half2 i holds
// channels i and i + 8.  A code in the low mantissa bits of 2^e, e such that they count ones, is 2^e + c.
__device__ __forceinline__ void unpack(uint32_t w, __half2 s, __half2 z, uint32_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i % 5, shift = 2 * (i - at);
    const uint32_t base = 0x6400u - (2u * at << 10);   // 2^(10 - 2 at)
    const uint32_t bits = ((w >> shift) & (0x00030003u << (2 * at))) | (base | base << 16);
    const __half2 one = __halves2half2(__ushort_as_half(base), __ushort_as_half(base));
    const __half2 v = __hfma2(__hsub2(*reinterpret_cast<const __half2*>(&bits), one), s, z);
    x[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

template <int GK, bool PAIR>
__global__ void __launch_bounds__(SC_THREADS, 1)
    chunk_scan_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ScanArgs A,
                      const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ uint8_t sc_raw[];
  ScanSmem& sm = *reinterpret_cast<ScanSmem*>(sc_raw + (-smem_u32(sc_raw) & 1023u));
  constexpr int NG = D / GK;
  constexpr int LAG = PAIR ? 1 : 2;   // steps between a tile's K and its V: a chain takes every LAG-th step
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SC_STAGES; ++s) {
      mbar_init(&sm.kv_full[s], 4);
      mbar_init(&sm.kv_empty[s], PAIR ? 2 : 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.s_full[a], 1);
      mbar_init(&sm.p_full[a][0], 4);
      mbar_init(&sm.p_full[a][1], 4);
      mbar_init(&sm.o_full[a], 1);
      mbar_init(&sm.o_empty[a], 4);
      mbar_init(&sm.turn[a], 1);
    }
    mbar_init_fence();
    prefetch_map(&q_map);
  }
  if (warp == SC_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  auto gave_up = [&]() { atomicOr(c.err, ERR_TIMEOUT); };
  const int per_tile = SC_ROWS >> A.lg;   // tokens of a tile of rows
  // tiles of rows of a segment's block
  auto row_tiles = [&](const Segment& s) {
    return PAIR && A.m[s.req] - s.block * 2 * per_tile > per_tile ? 2 : 1;
  };

  if (warp >= SC_MMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SC_OTHER_REGS));
    if (warp == SC_LOAD_WARP) {
      // ---- queries
      if (lane == 0) {
        bool ok = true;
        int loads = 0;
        Walk w = Walk::begin(A);
        for (; ok && w.next(A); w.done(A)) {
          if (loads > 0) ok = mbar_wait(&sm.q_empty, (loads - 1) & 1);
          if (!ok) break;
          const int tiles = row_tiles(w.s);
          mbar_expect_tx(&sm.q_full, tiles * TILE_BYTES);
          for (int a = 0; a < tiles; ++a)
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sm.q[a] + h * (TILE_BYTES / 2), &q_map, 64 * h, w.s.head * A.G,
                          A.row[w.s.req] + (w.s.block * (PAIR ? 2 : 1) + a) * per_tile, &sm.q_full);
          ++loads;
        }
        if (!ok) gave_up();
        // nothing may arrive after the CTA
        if (loads > 0) {
          mbar_wait(&sm.q_full, (loads - 1) & 1);
          if (ok) mbar_wait(&sm.q_empty, (loads - 1) & 1);
        }
      }
    } else if (warp < SC_LOAD_WARP) {
      // ---- products of chain a
      const int a = warp - SC_MMA_WARP;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { ok = mbar_wait_warp(bar, parity, ok); };
      const uint64_t q = desc_kmajor(smem_u32(sm.q[PAIR ? a : 0])), k_desc = desc_kmajor(smem_u32(sm.kv[0][1])),
                     v_desc = desc_nmajor(smem_u32(sm.kv[0][0]));
      const uint32_t s_col = 128 * a, o_col = 256 + 128 * a;
      int step = 0, segs = 0, tile = 0, outs = 0, batch = 0;
      Walk w = Walk::begin(A);
      for (; ok && w.next(A); w.done(A), ++segs) {
        const int n = w.s.j1 - w.s.j0;
        const bool two = PAIR && row_tiles(w.s) == 2;
        if (PAIR && a > 0 && !two) {   // no rows: only free the stages and the queries
          for (int i = 0; i < n + LAG && ok; ++i, ++step) {
            wait(&sm.kv_full[step % SC_STAGES], (step / SC_STAGES) & 1);
            if (ok) mbar_arrive_elected(&sm.kv_empty[step % SC_STAGES]);
          }
          if (ok) mbar_arrive_elected(&sm.q_empty);
          continue;
        }
        wait(&sm.q_full, segs & 1);
        bool first = true;   // of this chain in the segment
        bool last_s = false; // the chain's last S is issued: the queries are free when it is done
        for (int i = 0; i < n + LAG && ok; ++i, ++step) {
          const int st = step % SC_STAGES;
          if (!PAIR && st != a) continue;
          wait(&sm.kv_full[st], (step / SC_STAGES) & 1);
          if (!ok) break;
          tc_fence_after();
          if (i >= LAG) {   // P V of tile i - LAG
            if (first && outs > 0) wait(&sm.o_empty[a], (outs - 1) & 1);   // the last segment's rows are out of O
            if (two && a + batch > 0) wait(&sm.turn[a], (a == 0 ? batch - 1 : batch) & 1);
            const uint64_t v = v_desc + st * (2 * TILE_BYTES >> 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              wait(&sm.p_full[a][h], tile & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int s = 4 * h; s < 4 * h + 4; ++s)   // 16 keys
                mma_ts(o_col, s_col + 64 * h + 8 * (s % 4), v + (2048 * s >> 4), IDESC_PV_F16, !first || s > 0);
            }
            if (!ok) break;
            first = false;
            ++tile;
          }
          if (i < n) {      // S of tile i
            const uint64_t k = k_desc + st * (2 * TILE_BYTES >> 4);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              if (s == 6 && two && i >= LAG) mbar_arrive_elected(&sm.turn[a ^ 1]);
              const uint64_t off = ((s >> 2) * (TILE_BYTES / 2) + (s & 3) * 32) >> 4;
              mma_ss(s_col, q + off, k + off, IDESC_QK_F16, s > 0);
            }
            mma_commit(&sm.s_full[a]);
          } else if (two) {
            mbar_arrive_elected(&sm.turn[a ^ 1]);
          }
          if (i >= LAG) batch += two;
          if (i >= LAG && i >= n) mma_commit(&sm.o_full[a]);   // the chain's last
          if (!last_s && i + LAG >= n) {
            last_s = true;
            mma_commit(&sm.q_empty);
          }
          mma_commit(&sm.kv_empty[st]);
        }
        if (!first) ++outs;
      }
      if (!ok && lane == 0) gave_up();
    }
  } else if (warp >= SC_UNPACK_WARP) {
    // ---- keys and values, a key a thread
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SC_UNPACK_REGS));
    const int r = threadIdx.x & (SC_KEYS - 1);
    // steps looked up ahead: where the key's record is (null: zeros) for K of a step; V of a tile takes
    // that of LAG steps before
    struct Ahead {
      Walk w;
      int i, n;
      bool some;
    };
    Ahead at;
    at.w = Walk::begin(A);
    at.some = at.w.next(A);
    at.i = 0;
    at.n = at.some ? at.w.s.j1 - at.w.s.j0 : 0;
    // one step ahead of the data: page ids, and what else the record's address needs
    struct Look {
      int page, head;   // page as the table has it
      bool some, live;  // a key; a step (not behind the end)
    };
    auto look = [&]() {
      Look l{0, 0, false, at.some};
      if (!at.some) return l;
      if (at.i < at.n) {
        const int t = (at.w.s.j0 + at.i) * SC_KEYS + r;
        if (t < A.hist[at.w.s.req]) {
          l.page = c.hist_pt[(size_t)A.slot[at.w.s.req] * c.max_pages + t / PAGE];
          l.head = at.w.s.head;
          l.some = true;
        }
      }
      if (++at.i == at.n + LAG) {
        at.w.done(A);
        at.some = at.w.next(A);
        at.i = 0;
        at.n = at.some ? at.w.s.j1 - at.w.s.j0 : 0;
      }
      return l;
    };
    struct Data {
      uint4 w[2];
      uint32_t meta[NG];
    };
    auto fetch = [&](const Look& l, int which) {
      Data d;
      d.w[0] = d.w[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int n = 0; n < NG; ++n) d.meta[n] = 0;
      if (l.some && (l.page < 0 || l.page >= c.n_int2_pages)) {
        atomicOr(c.err, ERR_INT2_PAGE);   // (zeros)
      } else if (l.some) {
        const uint8_t* rec = int2_record(c, A.layer, l.page, l.head);
        const uint4* code = reinterpret_cast<const uint4*>(rec + (which ? V_CODES_OFF : K_CODES_OFF) + (r % PAGE) * CODE_BYTES);
        d.w[0] = code[0];
        d.w[1] = code[1];
        const uint32_t* m = reinterpret_cast<const uint32_t*>(
            rec + (which ? v_meta_off_for(GK) : k_meta_off_for(GK)) + (r % PAGE) * meta_bytes_for(GK));
#pragma unroll
        for (int n = 0; n < NG; ++n) d.meta[n] = m[n];
      }
      return d;
    };
    auto put = [&](uint8_t* tile, const Data& d) {
      const uint32_t w[8] = {d.w[0].x, d.w[0].y, d.w[0].z, d.w[0].w, d.w[1].x, d.w[1].y, d.w[1].z, d.w[1].w};
      const __half2 half = __float2half2_rn(0.5f);
      __half2 s, z;
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        if (p % (8 / NG) == 0) {
          const uint32_t m = d.meta[p / (8 / NG)], lo = m & 0xffff, hi = m >> 16;
          const uint32_t ss = lo | lo << 16, zz = hi | hi << 16;
          s = __hmul2(*reinterpret_cast<const __half2*>(&ss), half);
          z = __hmul2(*reinterpret_cast<const __half2*>(&zz), half);
        }
        uint32_t x[8];
        unpack(w[p], s, z, x);
        *reinterpret_cast<uint4*>(tile + tile_at(r, 2 * p)) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4*>(tile + tile_at(r, 2 * p + 1)) = make_uint4(x[4], x[5], x[6], x[7]);
      }
    };
    bool ok = true;
    const Look none{0, 0, false, true};
    Look back[LAG];                     // K's records of the LAG steps before
#pragma unroll
    for (int i = 0; i < LAG; ++i) back[i] = none;
    Look now = look(), next = look();
    Data k = fetch(now, 0), v = fetch(none, 1);
    for (int step = 0; now.live; ++step) {
      const int st = step % SC_STAGES;
      if (step >= SC_STAGES) ok = mbar_wait_warp(&sm.kv_empty[st], (step / SC_STAGES - 1) & 1, ok);
      if (!ok) break;
      const Data k_now = k, v_now = v;
      // what this step's record was for K is, LAG steps on, V's
#pragma unroll
      for (int i = LAG - 1; i > 0; --i) back[i] = back[i - 1];
      back[0] = now;
      k = fetch(next, 0);
      v = fetch(back[LAG - 1], 1);
      now = next;
      next = look();
      put(sm.kv[st][0], v_now);
      put(sm.kv[st][1], k_now);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.kv_full[st]);
    }
    if (!ok && lane == 0) gave_up();
  } else {
    // ---- softmax of chain a, one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SC_SOFTMAX_REGS));
    const int a = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = lane_off + 128 * a, to = lane_off + 256 + 128 * a;
    bool ok = true;
    int tile = 0, outs = 0, step0 = 0;   // key tiles and segments of this chain so far; steps of the CTA
    Walk w = Walk::begin(A);
    for (; ok && w.next(A); w.done(A)) {
      const Segment& s = w.s;
      const int n = s.j1 - s.j0, from = PAIR ? 0 : (a ^ step0) & 1;   // the chain's first tile
      step0 += n + LAG;
      if (PAIR && a >= row_tiles(s)) continue;
      const int m = A.m[s.req], tok0 = (s.block * (PAIR ? 2 : 1) + (PAIR ? a : 0)) * per_tile, tok = tok0 + (r >> A.lg);
      const int row = A.row[s.req] + min(tok, m - 1);
      const float scale2 = A.scale2 * A.q_scale[(size_t)row * A.Hq + s.head * A.G + (r & (A.G - 1))];
      const int hist = A.hist[s.req];
      float mx = NEG_INF, l = 0.0f;
      bool any = false;
      for (int i = from; i < n; i += LAG, ++tile) {
        ok = mbar_wait_warp(&sm.s_full[a], tile & 1, ok);
        if (!ok) break;
        tc_fence_after();
        const int left = hist - (s.j0 + i) * SC_KEYS;   // keys of the tile, at least one
        float t[4] = {NEG_INF, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[64];
          tmem_ld32(ts + 64 * h, x);
          tmem_ld32(ts + 64 * h + 32, x + 32);
          tc_wait_ld();
          if (left < SC_KEYS) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (64 * h + j >= left) x[j] = __float_as_uint(NEG_INF);
          }
#pragma unroll
          for (int j = 0; j < 64; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              t[k] = max3(t[k], __uint_as_float(x[j + 2 * k]), __uint_as_float(x[j + 2 * k + 1]));
        }
        const float top = fmaxf(max3(t[0], t[1], t[2]), t[3]) * scale2;
        const bool raise = top > mx + SC_LAZY || (mx == NEG_INF && top > NEG_INF);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? (mx == NEG_INF ? 0.0f : ex2f(mx - top)) : 1.0f;
          l *= f;
          if (raise) mx = top;
          if (any) {   // the product before S is done: S was issued after it
#pragma unroll 1
            for (int col = 0; col < 128; col += 16) {
              uint32_t o[16];
              tmem_ld16(to + col, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st16(to + col, o);
            }
          }
        }
        any = true;
        const float ref = mx == NEG_INF ? 0.0f : SC_SHIFT - mx;
        const float2 scale_2 = make_float2(scale2, scale2), ref_2 = make_float2(ref, ref);
        float2 sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t x[32], pk[16];
          tmem_ld32(ts + 32 * h, x);
          tc_wait_ld();
          if (left < SC_KEYS) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * h + j >= left) x[j] = __float_as_uint(NEG_INF);
          }
          float2 y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            y[j] = fma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), scale_2, ref_2);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            y[j].x = ex2f(y[j].x);
            y[j].y = ex2f(y[j].y);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            pk[j] = f16x2(y[j].x, y[j].y);
            sum[j & 3] = add2(sum[j & 3], y[j]);
          }
          tmem_st16(ts + 64 * (h / 2) + 16 * (h % 2), pk);   // P lies over S
          if (h == SC_FIRST / 32 - 1 || h == 3) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[a][h == 3]);
          }
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
      }
      if (!ok) break;
      // the rows' sums, maximum and sum to the workspace
      const int warp_tok = tok0 + (32 * (warp & 3) >> A.lg);
      if (any) {
        ok = mbar_wait_warp(&sm.o_full[a], outs & 1, ok);
        if (!ok) break;
        tc_fence_after();
        ++outs;
      }
      if (warp_tok < m) {
        float* part = A.records + ((size_t)(s.index + blockIdx.x) * 2 + a) * SC_ROWS * PARTIAL_FLOATS;
        part[r * PARTIAL_FLOATS + PARTIAL_M] = mx - SC_SHIFT;
        part[r * PARTIAL_FLOATS + PARTIAL_L] = l;
        uint8_t* stage = sm.out[warp];
#pragma unroll 1
        for (int col = 0; col < 128; col += 32) {
          uint32_t o[32];
          if (any) {
            tmem_ld32(to + col, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          __syncwarp();
#pragma unroll 4
          for (int k = 0; k < 8; ++k) {
            const int rw = 4 * k + lane / 8, rr = 32 * (warp & 3) + rw;
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rw * 128 + (((lane & 7) ^ (rw & 7)) << 4));
            if (tok0 + (rr >> A.lg) < m)
              *reinterpret_cast<uint4*>(part + rr * PARTIAL_FLOATS + col + 4 * (lane & 7)) = v;
          }
          __syncwarp();
        }
      }
      if (any) {   // O is read: the next segment may write it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty[a]);
      }
    }
    if (!ok && lane == 0) gave_up();
  }
  __syncwarp();
  __syncthreads();
  if (warp == SC_MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(0u) : "memory");
  }
}

// ---- queries in the rotated basis, and the merge ---------------------------------
constexpr int PITCH = D + 8;   // bf16 elements of a row in shared memory: ldmatrix without conflicts
constexpr int MG_THREADS = 256;

// Position 16 k + 2 i + b of a row that unpack() orders holds channel 16 k + 8 b + i.
__device__ __forceinline__ int channel_at(int pos) { return (pos & ~15) + 8 * (pos & 1) + ((pos >> 1) & 7); }

// A rotation (rows: outputs) as two bf16 parts, its columns as they are or in unpack()'s order.
struct Parts {
  alignas(16) uint16_t hi[D][PITCH], lo[D][PITCH];
};
template <bool ORDERED>
__device__ __forceinline__ void split_rotation(const float* m, Parts& s) {
#pragma unroll 4
  for (int i = threadIdx.x; i < D * (D / 16); i += MG_THREADS) {
    const int n = i / (D / 16), p = i % (D / 16);
    float f[16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(f + 4 * j) = reinterpret_cast<const float4*>(m + (size_t)n * D + 16 * p)[j];
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = ORDERED ? f[j] : f[2 * j], b = ORDERED ? f[j + 8] : f[2 * j + 1];
      hi[j] = bf16x2(a, b);
      lo[j] = bf16x2(a - __uint_as_float(hi[j] << 16), b - __uint_as_float(hi[j] & 0xffff0000u));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      *reinterpret_cast<uint4*>(&s.hi[n][16 * p + 8 * j]) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      *reinterpret_cast<uint4*>(&s.lo[n][16 * p + 8 * j]) = make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
  }
}
// acc += a b^T for MT tiles of 16 rows of a and this warp's 16 rows of b.
template <int MT>
__device__ __forceinline__ void multiply_rows(float (&acc)[MT][2][4], const uint16_t (*a)[PITCH], const uint16_t (*b)[PITCH]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    uint32_t bf[4];
    ldsm4(bf, smem_u32(&b[16 * warp + (lane & 7) + 8 * (lane >> 4)][16 * s + 8 * ((lane >> 3) & 1)]));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      uint32_t af[4];
      ldsm4(af, smem_u32(&a[16 * i + (lane & 15)][16 * s + 8 * (lane >> 4)]));
      mma_bf16(acc[i][0], af, bf[0], bf[1]);
      mma_bf16(acc[i][1], af, bf[2], bf[3]);
    }
  }
}

template <int MT>
struct RotateSmem {
  Parts r;
  alignas(16) uint16_t q[16 * MT][PITCH];
  alignas(16) float x[16 * MT][D + 4];
};
// 16 MT rows -- (token, head of the group), whatever requests they are of -- of one kv head.
template <int MT>
__global__ void __launch_bounds__(MG_THREADS)
    rotate_queries_kernel(const __grid_constant__ DevCache c, const __grid_constant__ RotateArgs A) {
  extern __shared__ __align__(16) uint8_t rt_raw[];
  RotateSmem<MT>& sm = *reinterpret_cast<RotateSmem<MT>*>(rt_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % c.Hkv;
  const int64_t row0 = (int64_t)(blockIdx.x / c.Hkv) * (16 * MT), rows = (int64_t)A.rows << A.lg;
  const int G = 1 << A.lg, Hq = G * c.Hkv;
  split_rotation<false>(c.rot_kt + ((size_t)A.layer * c.Hkv + head) * D * D, sm.r);   // (before the grid's dependency)
  grid_dep_launch();
  grid_dep_wait();
#pragma unroll
  for (int u = 0; u < MT; ++u) {
    const int r = 16 * u + threadIdx.x / 16, p = threadIdx.x % 16;
    const int64_t row = row0 + r;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rows)
      v = reinterpret_cast<const uint4*>(A.q + (row >> A.lg) * A.q_stride + (size_t)(head * G + (row & (G - 1))) * D)[p];
    *reinterpret_cast<uint4*>(&sm.q[r][8 * p]) = v;
  }
  __syncthreads();
  float acc[MT][2][4] = {};
  multiply_rows<MT>(acc, sm.q, sm.r.lo);
  multiply_rows<MT>(acc, sm.q, sm.r.hi);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(&sm.x[16 * i + lane / 4 + 8 * h][16 * warp + 8 * n + 2 * (lane & 3)]) =
            make_float2(acc[i][n][2 * h], acc[i][n][2 * h + 1]);
  __syncthreads();
#pragma unroll 2
  for (int r = warp; r < 16 * MT && row0 + r < rows; r += 8) {
    float y[4], top = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = sm.x[r][channel_at(4 * lane + j)];
      top = fmaxf(top, fabsf(y[j]));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    // 2^e with 2^10 <= top 2^e < 2^11, so that what falls below fp16's normal values is below 2^-24 of the row's largest
    const int e = min(max(137 - static_cast<int>(__float_as_uint(top) >> 23), -100), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23), down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const int64_t row = row0 + r;
    const size_t at = (size_t)(row >> A.lg) * Hq + head * G + (row & (G - 1));
    reinterpret_cast<uint2*>(A.out + at * D)[lane] = make_uint2(f16x2(y[0] * up, y[1] * up), f16x2(y[2] * up, y[3] * up));
    if (lane == 0) A.scale[at] = down;
  }
}

template <int ROWS>
struct MergeSmem {
  static constexpr int MT = ROWS > 16 ? ROWS / 16 : 1;
  Parts r;
  alignas(16) uint16_t hi[16 * MT][PITCH], lo[16 * MT][PITCH];   // the history's sums over the weights'
  alignas(16) float near[16 * MT][D + 4];                        // the other tokens'
  alignas(16) float part[8][2][D];                               // a warp's sums, where two warps share a row
  float m[8], l[8];
};
// ROWS rows of one request and kv head: partial rows of the scan's CTAs and of the BF16 tokens,
// each weighed with its maximum; two warps a row where there are four rows.
template <int ROWS, bool PAIR>
__global__ void __launch_bounds__(MG_THREADS)
    chunk_merge_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ScanArgs A,
                       const __grid_constant__ MergeArgs B) {
  extern __shared__ __align__(16) uint8_t mg_raw[];
  using Smem = MergeSmem<ROWS>;
  Smem& sm = *reinterpret_cast<Smem*>(mg_raw);
  constexpr int MT = Smem::MT, SHARE = ROWS < 8 ? 8 / ROWS : 1;   // warps of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x % c.Hkv, chunk = blockIdx.x / c.Hkv;
  split_rotation<true>(c.rot_v + ((size_t)A.layer * c.Hkv + head) * D * D, sm.r);   // (before the grid's dependency)
  int ri = 0, hi = A.n;
  while (hi - ri > 1) {
    const int mid = (ri + hi) >> 1;
    if (B.chunk[mid] <= chunk) ri = mid; else hi = mid;
  }
  const int row0 = (chunk - B.chunk[ri]) * ROWS, rows = A.m[ri] << A.lg;   // rows of the request and kv head
  if (ROWS < 16)   // the product takes 16 rows
    for (int i = threadIdx.x; i < 16 * PITCH / 8; i += MG_THREADS)
      reinterpret_cast<uint4*>(sm.hi)[i] = reinterpret_cast<uint4*>(sm.lo)[i] = make_uint4(0, 0, 0, 0);
  grid_dep_launch();
  grid_dep_wait();
  __syncthreads();
  const int64_t each = A.tiles[ri] + A.setup;
  for (int r = warp / SHARE; r < ROWS; r += 8 / SHARE) {
    const int rr = row0 + r;
    float4 far = make_float4(0, 0, 0, 0), near = far;
    float top = NEG_INF, l = 0.0f;
    if (rr < rows) {
      constexpr int BLOCK = PAIR ? 2 * SC_ROWS : SC_ROWS;
      const int64_t k = (int64_t)head * A.blocks[ri] + rr / BLOCK, start = A.cost[ri] + k * each;
      const int64_t c0 = chunk_of(A, start + A.setup), c1 = chunk_of(A, start + each - 1);
      // record j of the row: of the scan's CTAs in turn, both chains of each unless they have rows of their own
      const float* scan = A.records + ((size_t)(A.segment[ri] + k + c0) * 2 + (PAIR ? rr % BLOCK / SC_ROWS : 0)) * SC_ROWS * PARTIAL_FLOATS +
                          (size_t)(rr % SC_ROWS) * PARTIAL_FLOATS;
      const int count = static_cast<int>(c1 - c0 + 1) * (PAIR ? 1 : 2);
      constexpr size_t STEP = (size_t)(PAIR ? 2 : 1) * SC_ROWS * PARTIAL_FLOATS;
      const int back = B.near_blocks - 1 - (B.near_start[ri] + rr / (2 * SC_ROWS));
      const float* bf = B.near + (((size_t)back * B.near_splits * c.Hkv + head) * (2 * SC_ROWS) + rr % (2 * SC_ROWS)) * PARTIAL_FLOATS;
      const size_t near_step = (size_t)c.Hkv * (2 * SC_ROWS) * PARTIAL_FLOATS;
      for (int j = lane; j < count; j += 32) top = fmaxf(top, scan[j * STEP + PARTIAL_M]);
      for (int j = lane; j < B.near_splits; j += 32) top = fmaxf(top, bf[j * near_step + PARTIAL_M]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      // (a row without a maximum goes the same way: a NaN query's sums are NaN)
      const float ref = top == NEG_INF ? 0.0f : top;
      const int mine = warp % SHARE;
#pragma unroll 4
      for (int j = mine; j < count; j += SHARE) {
        const float* p = scan + j * STEP;
        const float f = ex2f(p[PARTIAL_M] - ref);
        const float4 v = reinterpret_cast<const float4*>(p)[lane];
        l = fmaf(p[PARTIAL_L], f, l);
        far.x = fmaf(v.x, f, far.x);
        far.y = fmaf(v.y, f, far.y);
        far.z = fmaf(v.z, f, far.z);
        far.w = fmaf(v.w, f, far.w);
      }
      for (int j = mine; j < B.near_splits; j += SHARE) {
        const float* p = bf + j * near_step;
        const float f = ex2f(p[PARTIAL_M] - ref);
        const float4 v = reinterpret_cast<const float4*>(p)[lane];
        l = fmaf(p[PARTIAL_L], f, l);
        near.x = fmaf(v.x, f, near.x);
        near.y = fmaf(v.y, f, near.y);
        near.z = fmaf(v.z, f, near.z);
        near.w = fmaf(v.w, f, near.w);
      }
    }
    if constexpr (SHARE > 1) {
      static_assert(SHARE == 2 && ROWS * SHARE == 8, "a row's two warps meet once");
      if (warp % SHARE) {
        reinterpret_cast<float4*>(sm.part[warp][0])[lane] = far;
        reinterpret_cast<float4*>(sm.part[warp][1])[lane] = near;
        if (lane == 0) sm.l[warp] = l;
      }
      __syncthreads();
      if (warp % SHARE) continue;
      const float4 x = reinterpret_cast<const float4*>(sm.part[warp + 1][0])[lane];
      const float4 y = reinterpret_cast<const float4*>(sm.part[warp + 1][1])[lane];
      far.x += x.x, far.y += x.y, far.z += x.z, far.w += x.w;
      near.x += y.x, near.y += y.y, near.z += y.z, near.w += y.w;
      l += sm.l[warp + 1];
    }
    // (values are halves of themselves in the scan)
    const float inv = l == 0.0f ? 0.0f : 1.0f / l, twice = 2.0f * inv;
    const float f[4] = {far.x * twice, far.y * twice, far.z * twice, far.w * twice};
    const uint32_t h0 = bf16x2(f[0], f[1]), h1 = bf16x2(f[2], f[3]);
    *reinterpret_cast<uint2*>(&sm.hi[r][4 * lane]) = make_uint2(h0, h1);
    *reinterpret_cast<uint2*>(&sm.lo[r][4 * lane]) =
        make_uint2(bf16x2(f[0] - __uint_as_float(h0 << 16), f[1] - __uint_as_float(h0 & 0xffff0000u)),
                   bf16x2(f[2] - __uint_as_float(h1 << 16), f[3] - __uint_as_float(h1 & 0xffff0000u)));
    *reinterpret_cast<float4*>(&sm.near[r][4 * lane]) = make_float4(near.x * inv, near.y * inv, near.z * inv, near.w * inv);
  }
  __syncthreads();
  float acc[MT][2][4] = {};
  multiply_rows<MT>(acc, sm.lo, sm.r.hi);
  multiply_rows<MT>(acc, sm.hi, sm.r.lo);
  multiply_rows<MT>(acc, sm.hi, sm.r.hi);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2* p = reinterpret_cast<float2*>(&sm.near[16 * i + lane / 4 + 8 * h][16 * warp + 8 * n + 2 * (lane & 3)]);
        const float2 y = *p;
        *p = make_float2(y.x + acc[i][n][2 * h], y.y + acc[i][n][2 * h + 1]);
      }
  __syncthreads();
  const int G = 1 << A.lg;
  for (int i = threadIdx.x; i < ROWS * 16; i += MG_THREADS) {
    const int r = i / 16, p = i % 16, rr = row0 + r;
    if (rr >= rows) continue;
    const float4 x = *reinterpret_cast<const float4*>(&sm.near[r][8 * p]), y = *reinterpret_cast<const float4*>(&sm.near[r][8 * p + 4]);
    uint16_t* out = B.out + ((size_t)(A.row[ri] + (rr >> A.lg)) * A.Hq + head * G + (rr & (G - 1))) * D;
    reinterpret_cast<uint4*>(out)[p] = make_uint4(bf16x2(x.x, x.y), bf16x2(x.z, x.w), bf16x2(y.x, y.y), bf16x2(y.z, y.w));
  }
}

// A kernel's shared memory (and, where it counts on them, registers), set once per device.
template <typename K>
cudaError_t set_up(K kernel, int bytes, int regs, std::atomic<unsigned>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 32 && (done.load() & (1u << dev)))) return e;
  if (regs) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != regs) return cudaErrorInvalidKernelImage;
  }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 32) done.fetch_or(1u << dev);
  return e;
}

template <int MT>
cudaError_t rotate(const DevCache& c, const RotateArgs& a, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(RotateSmem<MT>));
  static std::atomic<unsigned> done;
  const cudaError_t e = set_up(rotate_queries_kernel<MT>, bytes, 0, done);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (((int64_t)a.rows << a.lg) + 16 * MT - 1) / (16 * MT);
  return launch_dependent(rotate_queries_kernel<MT>, static_cast<unsigned>(chunks * c.Hkv), MG_THREADS, bytes, s, c, a);
}
template <int GK, bool PAIR>
cudaError_t scan(const DevCache& c, const ScanArgs& a, const CUtensorMap& q_map, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(ScanSmem)) + 1024;
  static std::atomic<unsigned> done;
  const cudaError_t e = set_up(chunk_scan_kernel<GK, PAIR>, bytes, SC_REGS, done);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_scan_kernel<GK, PAIR>, static_cast<unsigned>(a.ctas), SC_THREADS, bytes, s, c, a, q_map);
}
template <int ROWS, bool PAIR>
cudaError_t merge(const DevCache& c, const ScanArgs& a, MergeArgs& b, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(MergeSmem<ROWS>));
  static std::atomic<unsigned> done;
  const cudaError_t e = set_up(chunk_merge_kernel<ROWS, PAIR>, bytes, 0, done);
  if (e != cudaSuccess) return e;
  int chunks = 0;
  for (int i = 0; i < a.n; ++i) {
    b.chunk[i] = chunks;
    chunks += ((a.m[i] << a.lg) + ROWS - 1) / ROWS;
  }
  return launch_dependent(chunk_merge_kernel<ROWS, PAIR>, static_cast<unsigned>(chunks * c.Hkv), MG_THREADS, bytes, s, c, a, b);
}

}  // namespace

cudaError_t launch_rotate_queries(const DevCache& c, const RotateArgs& a, int sms, cudaStream_t s) {
  // rows of a CTA: 64, where that leaves every SM some, since each CTA splits a rotation of its own
  return (((int64_t)a.rows << a.lg) * c.Hkv >= (int64_t)sms * 64) ? rotate<4>(c, a, s) : rotate<1>(c, a, s);
}
cudaError_t launch_chunk_scan(const DevCache& c, const ScanArgs& a, bool pair, const CUtensorMap& q_map, cudaStream_t s) {
  if (c.gk == 64) return pair ? scan<64, true>(c, a, q_map, s) : scan<64, false>(c, a, q_map, s);
  return pair ? scan<128, true>(c, a, q_map, s) : scan<128, false>(c, a, q_map, s);
}
cudaError_t launch_chunk_merge(const DevCache& c, const ScanArgs& a, MergeArgs& b, bool pair, int sms, cudaStream_t s) {
  int64_t rows = 0;
  for (int i = 0; i < a.n; ++i) rows += (int64_t)a.m[i] << a.lg;
  rows *= c.Hkv;
  if (pair) return rows >= (int64_t)sms * 64 ? merge<64, true>(c, a, b, s) : merge<16, true>(c, a, b, s);
  // few rows have many records: four rows a CTA spread them
  return rows >= (int64_t)sms * 16 ? merge<16, false>(c, a, b, s) : merge<4, false>(c, a, b, s);
}

}  // namespace oscar
