// Attention of a chunk of new tokens of each request over the three-segment cache and, causally,
// over the chunk itself ("TogetherAI开源OSCAR" (ModelScope), section "OSCAR的设计": unpack, scale and
// zero, online-softmax merge of the segments; "Together AI Open-Sources OSCAR" (MarkTechPost),
// section "The Serving System").  Four kernels:
//   rotate_*_kernel        q R_K in fp16, each row scaled by a power of two, its channels in the
//                          order that unpacking leaves the codes in;
//   chunk_scan_kernel      the history: partial rows (unnormalised sums, maximum, sum);
//   paged_prefill_kernel   the BF16 tokens and the new ones, likewise (paged_prefill_device.cuh);
//   chunk_merge_*_kernel   their sum, the history's times R_V^T, over the weights' sum.
//
// chunk_scan_kernel: a CTA takes 128 keys at a time.  Four warps unpack them, a key a thread,
// into fp16 values z + s c in shared memory (off by 2^-11 of them and 2^-15 of the tile's largest), a tile's
// keys times 2^-a and its values times 2^-b: powers of two from their largest that keep them in range.  Per key
// tile and chain
//   S = Q K^T            128 x 128 x 128, tcgen05.mma, both operands in shared memory
//   p = exp2(S scale 2^a + b - m + 11)   one thread per row; fp16 (2^-11; the shift keeps weights down to
//                        2^-25 of the row's largest in full, where fp16 alone would flush them)
//   O = O + P V          tcgen05.mma, P from TMEM, O in TMEM
// with m the running maximum of the exponents with b, so of what a key adds to O; the weights' sum takes
// p 2^-b.
// The two chains are two tiles of 128 query rows (a row being a (token, head of the group) pair)
// that share every key, or, where a kv head has 128 rows or fewer, every other key tile each of
// the one tile of queries: a chain by itself is S, softmax, PV one after another.  Where 64 rows or
// fewer leave half of the softmax's warps idle, those unpack the values, the other four the keys
// (5 tokens over 100K: 62 us, 67.5 without).
//
// Bytes of history are few (72 a token-head).  With two tiles of rows a key tile moves 300 KB through
// shared memory -- operands 192, unpacked values 64, packed data 45 -- or 2350 cycles, and is 2048 of the tensor
// core's; it takes 3050 (tensor pipe 66 %).  2048 tokens over 60K, 32 heads of 8: 1258 us, 1.63 PFLOP/s.  With few
// rows it is bound by its copies (2 KB and less) and the barriers around them: 5 tokens over 100K 59 us, of which 46
// here, 0.39 us per 1K tokens.  Work is a line of key tiles, segment by segment -- (request, kv head, 256 rows) --
// with some set-up units in front of each, cut into one equal range per SM: a long request is spread over all of
// them, and none waits for the last segment.
#include <atomic>
#include <type_traits>

#include "append_device.cuh"
#include "chunk.h"
#include "values_device.cuh"

namespace oscar {
namespace {

using namespace paged;

constexpr int SC_THREADS = 512;                // softmax of chain 0, of chain 1, unpacking, the others
constexpr int SC_UNPACK_WARP = 8, SC_MMA_WARP = 12, SC_SIZE_WARP = 14, SC_FETCH_WARP = 15;
// Registers a thread: 128 at launch, then 168 for the softmax's two warpgroups, which hold a row
// of logits each, and 88 for the other two.
constexpr int SC_REGS = 128, SC_SOFTMAX_REGS = 168, SC_OTHER_REGS = 88;
static_assert(2 * SC_SOFTMAX_REGS + 2 * SC_OTHER_REGS <= 4 * SC_REGS, "a split above the launch's registers waits forever");
constexpr int SC_STAGES = 2;                   // of V of a key tile and K of the next
constexpr int SC_ROWS = 128, SC_KEYS = 128;
constexpr int SC_FEW = 64;                     // rows of which a chain's first two warps have the softmax
// Steps whose tiles' exponents are kept: those of step s are written when its packed data is there, so SLOTS + 2
// steps after the products of an earlier step were done.  P V of a tile, which awaits the weights that were made of
// its exponents, comes LAG steps after them: SLOTS + 2 + LAG steps have to be kept, 9 at most.
constexpr int SIZES = 16;
constexpr float SC_LAZY = 4.0f;                // the softmax reference moves only when exceeded by 2^4
// |S| is at most 128 x 2^11 x 2^-8.  Up to this scale logits stay within 2^22, where the roundings of a product, of the
// maximum and of the reference, 2^-2 each, leave a weight below 2^16.  Beyond it S is taken as differences to the row's
// largest of the tile, before the scale, so that logits of any size keep their order over tiles and segments.
constexpr float SC_STEEP = 0x1p12f;
constexpr float SC_STEEPEST = 0x1p117f;        // (so that a logit is finite)
constexpr float SC_SHIFT = 11.0f;              // weights are at most 2^15, and fp16's steps below 2^-14 cost nothing

// Packed data of a step: K codes of a tile, V codes of an earlier one and their {s, z}; {s, z} of the tile's own keys
// and values, page by page as records have them.
template <int GK>
struct Raw {
  static constexpr int META = SC_KEYS * meta_bytes_for(GK);
  alignas(16) uint8_t code[2][SC_KEYS * CODE_BYTES];
  alignas(16) uint8_t v_meta[META];
  alignas(16) uint8_t meta[2][META];
};
template <int GK, bool PAIR>
struct alignas(1024) ScanSmem {
  // steps of packed data in flight; where one tile of queries is enough, also in the other's place
  static constexpr int SLOTS = PAIR ? 2 : 2 + static_cast<int>(TILE_BYTES / sizeof(Raw<GK>));
  alignas(1024) uint8_t q[2][TILE_BYTES];                // two halves of 64 channels, [128 rows][128 B] swizzled
  alignas(1024) uint8_t kv[SC_STAGES][2][TILE_BYTES];    // V of an earlier key tile, K of this one
  alignas(128) Raw<GK> raw[2];
  alignas(16) uint8_t out[8][32 * 32];                   // per softmax warp: 32 bytes of its 32 rows
  alignas(16) float4 size[SIZES];                        // of a key tile: b, 2^a, 2^-b, 2^-a
  uint64_t size_full[SIZES];
  uint64_t q_full, q_empty, kv_full[SC_STAGES], kv_empty[SC_STAGES], raw_full[SLOTS], raw_empty[SLOTS];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_empty[2], turn[2];
  uint32_t tmem;
  __device__ Raw<GK>& slot(int i) {
    return i < 2 ? raw[i] : reinterpret_cast<Raw<GK>*>(q[1])[i - 2];
  }
};
static_assert(sizeof(ScanSmem<64, true>) + 1024 <= 232448 && sizeof(ScanSmem<64, false>) + 1024 <= 232448 &&
                  sizeof(ScanSmem<128, false>) + 1024 <= 232448,
              "shared memory of a CTA");


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

// A wait of a warp that is ahead of the others: one lane asks (all 32 of them asking all along slow the others'
// shared memory: 2K tokens over 60K cached 1400 us, 1286 this way; for waits that are short this one is slower).
__device__ __forceinline__ bool mbar_wait_lane(uint64_t* bar, uint32_t parity, bool ok) {
  if (!ok) return false;
  int done = 1;
  if ((threadIdx.x & 31) == 0) done = mbar_wait(bar, parity);
  done = __shfl_sync(0xffffffffu, done, 0);
  __syncwarp();
  return done != 0;
}
template <int GK, bool PAIR, bool FEW>
__global__ void __launch_bounds__(SC_THREADS, 1)
    chunk_scan_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ScanArgs A,
                      const __grid_constant__ CUtensorMap q_map) {
  extern __shared__ uint8_t sc_raw[];
  using Smem = ScanSmem<GK, PAIR>;
  Smem& sm = *reinterpret_cast<Smem*>(sc_raw + (-smem_u32(sc_raw) & 1023u));
  constexpr int NG = D / GK, SLOTS = Smem::SLOTS;
  constexpr int LAG = PAIR ? 1 : 2;   // steps between a tile's K and its V: a chain takes every LAG-th step
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SC_STAGES; ++s) {
      mbar_init(&sm.kv_full[s], FEW ? 8 : 4);
      mbar_init(&sm.kv_empty[s], PAIR ? 2 : 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&sm.raw_full[s], 1);
      mbar_init(&sm.raw_empty[s], FEW ? 8 : 4);
    }
    for (int s = 0; s < SIZES; ++s) mbar_init(&sm.size_full[s], 1);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.s_full[a], 1);
      mbar_init(&sm.p_full[a][0], 4);
      mbar_init(&sm.p_full[a][1], 4);
      mbar_init(&sm.o_full[a], 1);
      mbar_init(&sm.o_empty[a], FEW ? 2 : 4);
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
  // The grid before in the stream is the near rows' kernel, on which nothing here depends: its CTAs let
  // this grid start only when what came before them, the rotated queries among it, is complete, and the
  // two run side by side.  What was written so lately is read past the L1 caches.  Waiting for it at the
  // end makes this grid's completion stand for both.
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  auto gave_up = [&]() { atomicOr(c.err, ERR_TIMEOUT); };
  const int per_tile = SC_ROWS >> A.lg;   // tokens of a tile of rows
  // tiles of rows of a segment's block
  auto row_tiles = [&](const Segment& s) {
    return PAIR && A.m[s.req] - s.block * 2 * per_tile > per_tile ? 2 : 1;
  };

  // keys' and values' values: thread r those of a tile's key r; what is 0 (V) and 1 (K) from u0 to u1
  auto unpack = [&](int r, int u0, int u1) {
    bool ok = true;
    int step = 0;
    Walk w = Walk::begin(A);
    for (; ok && w.next(A); w.done(A)) {
      const int n = w.s.j1 - w.s.j0, left = A.hist[w.s.req] - w.s.j0 * SC_KEYS - r;   // keys from this thread's of tile 0 on
      for (int i = 0; i < n + LAG && ok; ++i, ++step) {
        const int st = step % SC_STAGES, at = step % SLOTS;
        const Raw<GK>& raw = sm.slot(at);
        ok = mbar_wait_warp(&sm.size_full[step % SIZES], (step / SIZES) & 1, ok);   // (behind the packed data)
        if (!ok) break;
        const bool now = i < n && i * SC_KEYS < left, then = i >= LAG && (i - LAG) * SC_KEYS < left;
        const float k_down = sm.size[step % SIZES].w, v_down = i >= LAG ? sm.size[(step - LAG) % SIZES].z : 0.0f;
        if (step >= SC_STAGES) ok = mbar_wait_warp(&sm.kv_empty[st], (step / SC_STAGES - 1) & 1, ok);
        if (!ok) break;
        // V of tile i - LAG, K of tile i (a loop: the code of four roles together is more than the instruction
        // caches hold)
#pragma unroll 1
        for (int u = u0; u < u1; ++u) {
          const float down = u ? k_down : v_down;
          const bool some = u ? now : then;
          // 32 bytes of codes, four lanes of eight the second half first: no two of them meet in a bank
          const uint4* code = reinterpret_cast<const uint4*>(raw.code[u ^ 1]) + 2 * r;
          const int turn = r >> 2 & 1;
          uint4 words[2] = {code[turn], code[turn ^ 1]};
          if (turn) {
            const uint4 swap = words[0];
            words[0] = words[1], words[1] = swap;
          }
          if (!some) words[0] = words[1] = make_uint4(0, 0, 0, 0);
          const uint32_t* meta = reinterpret_cast<const uint32_t*>(u ? raw.meta[r / PAGE] : raw.v_meta) + NG * (u ? r % PAGE : r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 64 channels
            uint8_t* to = sm.kv[st][u] + h * (TILE_BYTES / 2) + r * 128;
            const uint32_t m = some ? meta[NG == 2 ? h : 0] : 0;
            __half2 s[5], z;
            value_steps(m, down, s, z);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint2 word = p ? make_uint2(words[h].z, words[h].w) : make_uint2(words[h].x, words[h].y);
              uint32_t x[8];
              unpack_values(word.x, s, z, x);
              *reinterpret_cast<uint4*>(to + (((4 * p) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<uint4*>(to + (((4 * p + 1) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
              unpack_values(word.y, s, z, x);
              *reinterpret_cast<uint4*>(to + (((4 * p + 2) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<uint4*>(to + (((4 * p + 3) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.kv_full[st]);
          mbar_arrive(&sm.raw_empty[at]);
        }
      }
    }
    if (!ok && lane == 0) gave_up();
  };
  // softmax of chain a, one thread per row
  auto softmax = [&]() {
    const int a = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = lane_off + 128 * a, to = lane_off + 256 + 128 * a;
    auto meet_chain = [&](bool mine) {   // a barrier of the chain's warps: whether all say yes
      int all;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.b32 %0, 1, 0, q;\n}"
          : "=r"(all)
          : "r"(static_cast<int>(mine)), "r"(a + 1), "n"(FEW ? SC_FEW : SC_ROWS)
          : "memory");
      return all != 0;
    };
    bool ok = true;
    int tile = 0, outs = 0, step0 = 0;   // key tiles and segments of this chain so far; steps of the CTA
    Walk w = Walk::begin(A);
    for (; ok && w.next(A); w.done(A)) {
      const Segment& s = w.s;
      const int n = s.j1 - s.j0, from = PAIR ? 0 : (a ^ step0) & 1;   // the chain's first tile
      int step = step0 + from;
      step0 += n + LAG;
      if (PAIR && a >= row_tiles(s)) continue;
      const int m = A.m[s.req], tok0 = (s.block * (PAIR ? 2 : 1) + (PAIR ? a : 0)) * per_tile, tok = tok0 + (r >> A.lg);
      const int row = A.row[s.req] + min(tok, m - 1);
      // (above 0, so that a masked key's -inf stays that; logits of below 2^30 times 2^-100 are 0 for exp2)
      const float scale2 = fmaxf(A.scale2 * __ldcg(A.q_scale + (size_t)row * A.Hq + s.head * A.G + (r & (A.G - 1))), 0x1p-100f);
      // warps of the tile that have rows; the first arrives for those without, which only meet the others behind the
      // segment: whatever their rows of P are, a row of O has the same row of P alone
      const int busy = min(4, (((m - tok0) << A.lg) + 31) / 32);
      const uint32_t arrivals = (warp & 3) == 0 ? 5 - busy : 1;
      const bool idle = (warp & 3) >= busy;
      int left = A.hist[s.req] - (s.j0 + from) * SC_KEYS;   // keys from the tile on
      float mx = NEG_INF, l = 0.0f;
      bool any = false;
      const int tiles = n > from ? (n - from + LAG - 1) / LAG : 0;   // of the chain
      if (idle) tile += tiles;
      auto keys = [&](auto any_scale) {   // the chain's key tiles; false: no row's scale is above SC_STEEP
        constexpr bool ANY_SCALE = decltype(any_scale)::value;
        for (int i = idle ? n : from; i < n; i += LAG, step += LAG, ++tile, left -= LAG * SC_KEYS) {
          ok = mbar_wait_warp(&sm.s_full[a], tile & 1, ok);
          if (!ok) break;
          tc_fence_after();
          // (written before the keys were unpacked, so before S)
          const float2 size = *reinterpret_cast<const float2*>(&sm.size[step % SIZES]);
          const float scale = fminf(scale2 * size.y, SC_STEEPEST);
          const bool steep = ANY_SCALE && scale > SC_STEEP;
          float zero = size.x;   // exponent of what S holds as 0
          if (ANY_SCALE && __any_sync(0xffffffffu, steep)) {   // a row's form depends on the row alone
            float most = NEG_INF;
#pragma unroll 1
            for (int col = 0; col < SC_KEYS; col += 16) {
              uint32_t o[16];
              tmem_ld16(ts + col, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (col + j < left) most = fmaxf(most, __uint_as_float(o[j]));
            }
            const float less = steep ? most : 0.0f;
#pragma unroll 1
            for (int col = 0; col < SC_KEYS; col += 16) {
              uint32_t o[16];
              tmem_ld16(ts + col, o);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) - less);
              tmem_st16(ts + col, o);
            }
            tc_wait_st();
            zero = fmaf(less, scale, size.x);
          }
          uint32_t xr[128];
#pragma unroll
          for (int h = 0; h < 4; ++h) tmem_ld32(ts + 32 * h, xr + 32 * h);
          tc_wait_ld();
          float* x = reinterpret_cast<float*>(xr);
          if (left < SC_KEYS) {   // keys behind the end
#pragma unroll
            for (int j = 0; j < SC_KEYS; ++j)
              if (j >= left) x[j] = NEG_INF;
          }
          float t[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = x[k];
#pragma unroll
          for (int j = 4; j < 124; j += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = max3(t[k], x[j + 2 * k], x[j + 2 * k + 1]);
          const float top = fmaf(fmaxf(max3(t[0], t[1], max3(t[2], t[3], x[124])), max3(x[125], x[126], x[127])), scale, zero);
          // (as a difference: it is exact near a large maximum, where mx + SC_LAZY may be rounded up by more than that)
          const bool raise = top - mx > SC_LAZY;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? (mx == NEG_INF ? 0.0f : ex2f(mx - top)) : 1.0f;
            l *= f;
            if (raise) mx = top;
            if (any) {   // the product before S is done: S was issued after it
#pragma unroll 1
              for (int col = 0; col < 128; col += 16) {   // in small pieces: the logits are live
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
          const float ref = steep ? (zero - mx) + SC_SHIFT : size.x + (mx == NEG_INF ? 0.0f : SC_SHIFT - mx);
          const float2 scale_2 = make_float2(scale, scale), ref_2 = make_float2(ref, ref);
          float2 sum[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) sum[k] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int h = 0; h < 4; ++h) {   // 32 keys
            float2 y[16];
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = fma2(make_float2(x[32 * h + 2 * j], x[32 * h + 2 * j + 1]), scale_2, ref_2);
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
            tmem_st16(ts + 64 * (h >> 1) + 16 * (h & 1), pk);   // P lies over S, 64 keys in 32 columns
            if (h & 1) {
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.p_full[a][h >> 1], arrivals);
            }
          }
          sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l = fmaf(sum[0].x + sum[0].y, sm.size[step % SIZES].z, l);
        }
      };
      if constexpr (PAIR) {
        // The head's threshold, which clips what is rotated, bounds 2^a (1 % and 2^-22 for the roundings of s and z).
        // A loop for rows that it keeps below: 2048 tokens over 60K 1319 us, 1345 with the other loop alone -- which is
        // the one where rows are few: 5 over 100K 59.1, 61.1 with both.  (Rows beyond SC_STEEP: 2186 and 80.)
        const float tau = c.tau_k[(size_t)A.layer * c.Hkv + s.head];
        const float most = pow2(value_exponent(__float_as_uint(fmaf(1.01f, tau, 0x1p-22f))));
        if (__any_sync(0xffffffffu, scale2 * most > SC_STEEP)) keys(std::true_type()); else keys(std::false_type());
      } else {
        keys(std::true_type());
      }
      // the rows' sums, maximum and sum to the workspace
      if (tiles > 0) {
        if (!idle) ok = mbar_wait_warp(&sm.o_full[a], outs & 1, ok);
        ok = meet_chain(ok);
        if (!ok) break;
        tc_fence_after();
        ++outs;
      }
      if (!idle) {
        float* part = A.records + ((size_t)(s.index + blockIdx.x) * 2 + a) * SC_ROWS * PARTIAL_FLOATS;
        part[r * PARTIAL_FLOATS + PARTIAL_M] = mx - SC_SHIFT;
        part[r * PARTIAL_FLOATS + PARTIAL_L] = l;
        uint8_t* stage = sm.out[warp];
#pragma unroll 1
        for (int col = 0; col < 128; col += 32) {
          uint32_t o[32];
          if (tiles > 0) {
            tmem_ld32(to + col, o);
            tc_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          }
          // turned through shared memory, so that two lanes store 32 bytes of a row together
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<uint4*>(stage + lane * 32 + ((k ^ (lane >> 2 & 1)) << 4)) =
                  make_uint4(o[8 * j + 4 * k], o[8 * j + 4 * k + 1], o[8 * j + 4 * k + 2], o[8 * j + 4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int rw = 16 * k + lane / 2, rr = 32 * (warp & 3) + rw;
              const uint4 v = *reinterpret_cast<const uint4*>(stage + rw * 32 + (((lane & 1) ^ (rw >> 2 & 1)) << 4));
              if (tok0 + (rr >> A.lg) < m)
                *reinterpret_cast<uint4*>(part + rr * PARTIAL_FLOATS + col + 8 * j + 4 * (lane & 1)) = v;
            }
            __syncwarp();
          }
        }
      }
      if (tiles > 0) {   // O is read: the next segment may write it
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty[a]);
      }
    }
    if (!ok && lane == 0) gave_up();
  };

  if (warp >= SC_MMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SC_OTHER_REGS));
    if (warp == SC_SIZE_WARP) {
      // ---- exponents of a tile's keys and values, four tokens a lane
      bool ok = true;
      int step = 0;
      Walk w = Walk::begin(A);
      for (; ok && w.next(A); w.done(A)) {
        const int n = w.s.j1 - w.s.j0;
        int left = A.hist[w.s.req] - w.s.j0 * SC_KEYS - lane;   // keys from this lane's first on
        for (int i = 0; i < n + LAG && ok; ++i, ++step, left -= SC_KEYS) {
          const int at = step % SLOTS;
          ok = mbar_wait_lane(&sm.raw_full[at], (step / SLOTS) & 1, ok);
          if (!ok) break;
          uint32_t top[2] = {0, 0};
          if (i < n) {
#pragma unroll 1
            for (int u = 0; u < 2; ++u) {
              const uint8_t* from = sm.slot(at).meta[0] + u * (Raw<GK>::META / 2);
              __half2 most = __float2half2_rn(0.0f);
#pragma unroll
              for (int k = 0; k < SC_KEYS / 32; k += 2 / NG) {   // two groups of a token, or two tokens
                const uint8_t* page = from + (k >> 1) * Raw<GK>::META;
                uint2 m;
                if constexpr (NG == 2) {
                  m = reinterpret_cast<const uint2*>(page)[32 * (k & 1) + lane];
                } else {
                  m = make_uint2(reinterpret_cast<const uint32_t*>(page)[lane], reinterpret_cast<const uint32_t*>(page)[32 + lane]);
                  if (32 * k + 32 >= left) m.y = 0;
                }
                if (32 * k >= left) m = make_uint2(0, 0);
                most = __hmax2(most, largest_values(m));
              }
              top[u] = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(__low2float(most), __high2float(most))));
            }
          }
          if (lane == 0) {
            const int a = value_exponent(top[0]), b = value_exponent(top[1]);
            sm.size[step % SIZES] = make_float4(static_cast<float>(b), pow2(a), pow2(-b), pow2(-a));
            mbar_arrive(&sm.size_full[step % SIZES]);
          }
        }
      }
      if (!ok && lane == 0) gave_up();
    } else if (warp == SC_FETCH_WARP) {
      // ---- queries, and packed keys and values: a lane a piece of a page; page ids are looked up 32 at a time, 16
      // steps ahead (a look-up a step, one step ahead: 200K tokens 104 us, 101 this way)
      static_assert(v_meta_off_for(GK) == k_meta_off_for(GK) + Raw<GK>::META / 2, "{s, z} of K and V side by side");
      const uint8_t* const pool = c.int2 + A.layer * c.int2_layer_stride;
      const size_t page_bytes = (size_t)c.Hkv * c.record;
      const int u = lane & 1, kind = lane >> 1;   // page of the tile; K codes, {s, z}, V codes and {s, z} of LAG steps ago
      const int lag = kind < 2 ? 0 : LAG, size = kind == 1 ? Raw<GK>::META : kind == 3 ? Raw<GK>::META / 2 : PAGE * CODE_BYTES;
      const int off = kind == 0 ? K_CODES_OFF : kind == 1 ? k_meta_off_for(GK) : kind == 2 ? V_CODES_OFF : v_meta_off_for(GK);
      const uint32_t to = u * size + static_cast<uint32_t>(kind == 0   ? offsetof(Raw<GK>, code)
                                                           : kind == 1 ? offsetof(Raw<GK>, meta)
                                                           : kind == 2 ? offsetof(Raw<GK>, code) + SC_KEYS * CODE_BYTES
                                                                       : offsetof(Raw<GK>, v_meta));
      bool ok = true;
      int step = 0, loads = 0;
      Walk w = Walk::begin(A);
      for (; ok && w.next(A); w.done(A)) {
        const int n = w.s.j1 - w.s.j0, pages = (A.hist[w.s.req] + PAGE - 1) / PAGE - 2 * w.s.j0, head = w.s.head;
        const int q_at = loads > 0;   // the queries come behind what can be fetched while the last segment's are in use
        const int32_t* table = c.hist_pt + (size_t)A.slot[w.s.req] * c.max_pages + 2 * w.s.j0;
        auto has = [&](int i) { return lane < 8 && i >= lag && i - lag < n && 2 * (i - lag) + u < pages; };
        auto look = [&](int first) { return first + lane < pages && first + lane < 2 * n ? __ldcg(table + first + lane) : 0; };
        int before = 0, ids = 0, next = look(0);   // of pages from 32 (i / 16 - 1), 32 (i / 16) and 32 (i / 16 + 1) on
        for (int i = 0; i < n + LAG; ++i, ++step) {
          if (i % 16 == 0) before = ids, ids = next, next = look(2 * i + 32);
          const int mine = 2 * (i - lag) + u, new_id = __shfl_sync(0xffffffffu, ids, mine), old_id = __shfl_sync(0xffffffffu, before, mine);
          int page = mine >> 5 == i >> 4 ? new_id : old_id;
          const int at = step % SLOTS;
          if (step >= SLOTS) ok = mbar_wait_lane(&sm.raw_empty[at], (step / SLOTS - 1) & 1, ok);
          if (!ok) break;
          const bool some = has(i);
          if (some && (page < 0 || page >= c.n_int2_pages)) {
            atomicOr(c.err, ERR_INT2_PAGE);
            page = 0;
          }
          const uint32_t bytes = __reduce_add_sync(0xffffffffu, some ? size : 0);
          if (lane == 0) mbar_expect_tx(&sm.raw_full[at], bytes);
          __syncwarp();
          if (some)
            tma_load_1d(reinterpret_cast<uint8_t*>(&sm.slot(at)) + to, pool + page * page_bytes + head * c.record + off, size,
                        &sm.raw_full[at]);
          if (i == q_at) {
            if (loads > 0) ok = mbar_wait_lane(&sm.q_empty, (loads - 1) & 1, ok);
            if (!ok) {
              ++step;
              break;
            }
            const int tiles = row_tiles(w.s);
            if (lane == 0) mbar_expect_tx(&sm.q_full, tiles * TILE_BYTES);
            __syncwarp();
            if (lane < 2 * tiles)
              tma_load_3d(sm.q[lane >> 1] + (lane & 1) * (TILE_BYTES / 2), &q_map, 64 * (lane & 1), head * A.G,
                          A.row[w.s.req] + (w.s.block * (PAIR ? 2 : 1) + (lane >> 1)) * per_tile, &sm.q_full);
            ++loads;
          }
        }
      }
      if (!ok && lane == 0) gave_up();
      // nothing may arrive after the CTA
      if (loads > 0) {
        mbar_wait(&sm.q_full, (loads - 1) & 1);
        if (ok) mbar_wait(&sm.q_empty, (loads - 1) & 1);
      }
      for (int k = max(0, step - SLOTS); k < step; ++k) mbar_wait(&sm.raw_full[k % SLOTS], (k / SLOTS) & 1);
    } else if (warp < SC_SIZE_WARP) {
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(SC_OTHER_REGS));
    unpack(threadIdx.x & (SC_KEYS - 1), FEW ? 1 : 0, 2);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SC_SOFTMAX_REGS));
    if (FEW && (warp & 2)) {
      unpack(64 * (warp >> 2) + 32 * (warp & 1) + lane, 0, 1);
    } else {
      softmax();
    }
  }
  __syncwarp();
  grid_dep_wait();
  __syncthreads();
  if (warp == SC_MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(0u) : "memory");
  }
}

// ---- queries in the rotated basis, and the merge ---------------------------------
constexpr int PITCH = D + 8;   // bf16 elements of a row in shared memory: ldmatrix without conflicts
constexpr int MG_THREADS = 256;

// A rotation (rows: outputs) as two bf16 parts.
struct Parts {
  alignas(16) uint16_t hi[D][PITCH], lo[D][PITCH];
};
__device__ __forceinline__ void split_rotation(const float* m, Parts& s) {
#pragma unroll 4
  for (int i = threadIdx.x; i < D * (D / 8); i += MG_THREADS) {
    const int n = i / (D / 8), p = i % (D / 8);
    float f[8];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4*>(f + 4 * j) = reinterpret_cast<const float4*>(m + (size_t)n * D + 8 * p)[j];
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = bf16x2(f[2 * j], f[2 * j + 1]);
      lo[j] = bf16x2(f[2 * j] - __uint_as_float(hi[j] << 16), f[2 * j + 1] - __uint_as_float(hi[j] & 0xffff0000u));
    }
    *reinterpret_cast<uint4*>(&s.hi[n][8 * p]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(&s.lo[n][8 * p]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
// 2^e with 2^10 <= top 2^e < 2^11, so that what falls below fp16's normal values is below 2^-24 of the row's largest.
__device__ __forceinline__ int row_exponent(float top) {
  return min(137 - static_cast<int>(__float_as_uint(top) >> 23), 126);
}

constexpr int UNIT = 16;       // rows of a warp's product
struct RotateSmem {
  Parts r;
  alignas(16) uint16_t q[8][UNIT][PITCH];
};
// A warp takes 16 rows -- (token, head of the group), whatever requests they are of -- of one
// kv head at a time; the CTA keeps that head's rotation.  (1216 tokens of 32 heads: 14.5 us by itself, most of it
// staging the rotation, which lies under the kernel before where there is one.)
__global__ void __launch_bounds__(MG_THREADS, 2)
    rotate_queries_kernel(const __grid_constant__ DevCache c, const __grid_constant__ RotateArgs A, int per_head) {
  extern __shared__ __align__(16) uint8_t rt_raw[];
  RotateSmem& sm = *reinterpret_cast<RotateSmem*>(rt_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int head = blockIdx.x / per_head, G = 1 << A.lg, Hq = G * c.Hkv;
  const int64_t rows = (int64_t)A.rows << A.lg;
  split_rotation(c.rot_kt + ((size_t)A.layer * c.Hkv + head) * D * D, sm.r);   // (before the grid's dependency)
  grid_dep_launch();
  grid_dep_wait();
  __syncthreads();
  uint16_t (*q)[PITCH] = sm.q[warp];
  for (int64_t row0 = ((int64_t)(blockIdx.x % per_head) + per_head * warp) * UNIT; row0 < rows; row0 += (int64_t)per_head * 8 * UNIT) {
    uint4 v[UNIT / 2];
#pragma unroll
    for (int u = 0; u < UNIT / 2; ++u) {
      const int64_t row = row0 + 2 * u + lane / 16;
      v[u] = make_uint4(0, 0, 0, 0);
      if (row < rows)
        v[u] = reinterpret_cast<const uint4*>(A.q + (row >> A.lg) * A.q_stride + (size_t)(head * G + (row & (G - 1))) * D)[lane % 16];
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < UNIT / 2; ++u) *reinterpret_cast<uint4*>(&q[2 * u + lane / 16][8 * (lane % 16)]) = v[u];
    __syncwarp();
    uint32_t a[8][4];
#pragma unroll
    for (int s = 0; s < 8; ++s) ldsm4(a[s], smem_u32(&q[lane & 15][16 * s + 8 * (lane >> 4)]));
    float x[16][4];
    float top[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = x[n + 1][i] = 0.0f;
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          uint32_t b[4];
          const uint16_t (*w)[PITCH] = part ? sm.r.hi : sm.r.lo;
          ldsm4(b, smem_u32(&w[8 * n + (lane & 7) + 8 * (lane >> 4)][16 * s + 8 * ((lane >> 3) & 1)]));
          mma_bf16(x[n], a[s], b[0], b[1]);
          mma_bf16(x[n + 1], a[s], b[2], b[3]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i / 2] = fmaxf(top[i / 2], fmaxf(fabsf(x[n][i]), fabsf(x[n + 1][i])));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // this thread's columns of row lane / 4 + 8 h
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      const int e = row_exponent(top[h]);
      const float up = pow2(e), down = pow2(-e);
      const int64_t row = row0 + lane / 4 + 8 * h;
      if (row >= rows) continue;
      const size_t at = (size_t)(row >> A.lg) * Hq + head * G + (row & (G - 1));
      // channels 16 k + 2 t, + 1, + 8, + 9 are positions 16 k + 4 t, + 2, + 1, + 3
#pragma unroll
      for (int k = 0; k < 8; ++k)
        reinterpret_cast<uint2*>(A.out + at * D)[4 * k + (lane & 3)] =
            make_uint2(f16x2(x[2 * k][2 * h] * up, x[2 * k + 1][2 * h] * up),
                       f16x2(x[2 * k][2 * h + 1] * up, x[2 * k + 1][2 * h + 1] * up));
      if ((lane & 3) == 0) A.scale[at] = down;
    }
  }
}

// Few rows: four of a CTA, which takes the rotation from the L2 cache straight into registers (a thread half a
// row of it), where staging it in shared memory would take longer than the rest.
constexpr int FEW = 4;
// y[r][n] = sum_k x[r][k] m[n][k], thread (n, half) having m's row n from 64 half on in f; the same sum in both.
template <int ROWS>
__device__ __forceinline__ void times_rotation(const float4 (&f)[16], const float (*x)[D], float (&y)[ROWS]) {
  const int half = threadIdx.x & 1;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(&x[r][64 * half + 4 * i]);
      s[0] = fmaf(f[i].x, v.x, s[0]);
      s[1] = fmaf(f[i].y, v.y, s[1]);
      s[0] = fmaf(f[i].z, v.z, s[0]);
      s[1] = fmaf(f[i].w, v.w, s[1]);
    }
    y[r] = s[0] + s[1];
    y[r] += __shfl_xor_sync(0xffffffffu, y[r], 1);
  }
}
__device__ __forceinline__ void take_rotation(float4 (&f)[16], const float* m) {
  const float4* row = reinterpret_cast<const float4*>(m + (size_t)(threadIdx.x >> 1) * D + 64 * (threadIdx.x & 1));
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = row[i];
}
// Where unpack_values() leaves channel c of a row.
__device__ __forceinline__ int position_of(int c) { return (c & ~15) + 2 * (c & 7) + (c >> 3 & 1); }

__global__ void __launch_bounds__(MG_THREADS)
    rotate_few_kernel(const __grid_constant__ DevCache c, const __grid_constant__ RotateArgs A) {
  __shared__ alignas(16) float x[FEW][D];
  __shared__ float top[FEW][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = threadIdx.x >> 1;
  const int head = blockIdx.x % c.Hkv, G = 1 << A.lg, Hq = G * c.Hkv;
  const int64_t row0 = (int64_t)(blockIdx.x / c.Hkv) * FEW, rows = (int64_t)A.rows << A.lg;
  float4 f[16];
  take_rotation(f, c.rot_kt + ((size_t)A.layer * c.Hkv + head) * D * D);   // (before the grid's dependency)
  grid_dep_launch();
  grid_dep_wait();
  for (int i = threadIdx.x; i < FEW * D / 2; i += MG_THREADS) {
    const int64_t row = row0 + i / (D / 2);
    uint32_t v = 0;
    if (row < rows)
      v = reinterpret_cast<const uint32_t*>(A.q + (row >> A.lg) * A.q_stride + (size_t)(head * G + (row & (G - 1))) * D)[i % (D / 2)];
    x[i / (D / 2)][2 * (i % (D / 2))] = __uint_as_float(v << 16);
    x[i / (D / 2)][2 * (i % (D / 2)) + 1] = __uint_as_float(v & 0xffff0000u);
  }
  __syncthreads();
  float y[FEW];
  times_rotation(f, x, y);
#pragma unroll
  for (int r = 0; r < FEW; ++r) {
    float t = fabsf(y[r]);
#pragma unroll
    for (int off = 16; off > 1; off >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
    if (lane == 0) top[r][warp] = t;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < FEW; ++r) {
    float t = top[r][0];
#pragma unroll
    for (int i = 1; i < 8; ++i) t = fmaxf(t, top[r][i]);
    const int e = row_exponent(t);
    const int64_t row = row0 + r;
    if (row >= rows || (threadIdx.x & 1)) continue;
    const size_t at = (size_t)(row >> A.lg) * Hq + head * G + (row & (G - 1));
    A.out[at * D + position_of(n)] = __half_as_ushort(__float2half_rn(y[r] * pow2(e)));
    if (n == 0) A.scale[at] = pow2(-e);
  }
}

// Rows of one request and kv head, the CTA's eight warps shared among them: partial rows of the scan's CTAs and of the
// BF16 tokens, each weighed with its maximum.
template <bool PAIR, int ROWS>
__global__ void __launch_bounds__(MG_THREADS)
    chunk_merge_few_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ScanArgs A,
                           const __grid_constant__ MergeArgs B) {
  constexpr int SHARES = 8 / ROWS;   // warps of a row
  __shared__ alignas(16) float far[ROWS][D], near[ROWS][D], part[ROWS][SHARES - 1][2][D];
  __shared__ float part_l[ROWS][SHARES - 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = threadIdx.x >> 1;
  const int head = blockIdx.x % c.Hkv, chunk = blockIdx.x / c.Hkv, G = 1 << A.lg;
  float4 f[16];
  take_rotation(f, c.rot_v + ((size_t)A.layer * c.Hkv + head) * D * D);   // (before the grid's dependency)
  int ri = 0, hi = A.n;
  while (hi - ri > 1) {
    const int mid = (ri + hi) >> 1;
    if (B.chunk[mid] <= chunk) ri = mid; else hi = mid;
  }
  const int row0 = (chunk - B.chunk[ri]) * ROWS, rows = A.m[ri] << A.lg;   // rows of the request and kv head
  const int r = warp / SHARES, share = warp % SHARES, rr = row0 + r;
  constexpr int BLOCK = PAIR ? 2 * SC_ROWS : SC_ROWS;
  const int64_t each = A.tiles[ri] + A.setup, k = (int64_t)head * A.blocks[ri] + rr / BLOCK, start = A.cost[ri] + k * each;
  const int64_t c0 = chunk_of(A, start + A.setup), c1 = chunk_of(A, start + each - 1);
  // record j of the row: of the scan's CTAs in turn, both chains of each unless they have rows of their own
  const float* scan = A.records + ((size_t)(A.segment[ri] + k + c0) * 2 + (PAIR ? rr % BLOCK / SC_ROWS : 0)) * SC_ROWS * PARTIAL_FLOATS +
                      (size_t)(rr % SC_ROWS) * PARTIAL_FLOATS;
  const int count = static_cast<int>(c1 - c0 + 1) * (PAIR ? 1 : 2);
  constexpr size_t STEP = (size_t)(PAIR ? 2 : 1) * SC_ROWS * PARTIAL_FLOATS;
  const int back = B.near_blocks - 1 - (B.near_start[ri] + rr / (2 * SC_ROWS));
  const float* bf = B.near + (((size_t)back * B.near_splits * c.Hkv + head) * (2 * SC_ROWS) + rr % (2 * SC_ROWS)) * PARTIAL_FLOATS;
  const size_t near_step = (size_t)c.Hkv * (2 * SC_ROWS) * PARTIAL_FLOATS;
  grid_dep_launch();
  grid_dep_wait();
  float4 x = make_float4(0, 0, 0, 0), y = x;
  float l = 0.0f;
  if (rr < rows) {
    float top = NEG_INF;
    for (int j = lane; j < count; j += 32) top = fmaxf(top, scan[j * STEP + PARTIAL_M]);
    for (int j = lane; j < B.near_splits; j += 32) top = fmaxf(top, bf[j * near_step + PARTIAL_M]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    // (a row without a maximum goes the same way: a NaN query's sums are NaN)
    const float ref = top == NEG_INF ? 0.0f : top;
    auto add = [&](const float* p, float4& to) {
      const float w = ex2f(p[PARTIAL_M] - ref);
      const float4 v = reinterpret_cast<const float4*>(p)[lane];
      l = fmaf(p[PARTIAL_L], w, l);
      to.x = fmaf(v.x, w, to.x);
      to.y = fmaf(v.y, w, to.y);
      to.z = fmaf(v.z, w, to.z);
      to.w = fmaf(v.w, w, to.w);
    };
#pragma unroll 4
    for (int j = share; j < count; j += SHARES) add(scan + j * STEP, x);
    for (int j = share; j < B.near_splits; j += SHARES) add(bf + j * near_step, y);
  }
  if (share) {
    reinterpret_cast<float4*>(part[r][share - 1][0])[lane] = x;
    reinterpret_cast<float4*>(part[r][share - 1][1])[lane] = y;
    if (lane == 0) part_l[r][share - 1] = l;
  }
  __syncthreads();
  if (!share) {
#pragma unroll
    for (int i = 0; i < SHARES - 1; ++i) {
      const float4 u = reinterpret_cast<const float4*>(part[r][i][0])[lane], v = reinterpret_cast<const float4*>(part[r][i][1])[lane];
      x.x += u.x, x.y += u.y, x.z += u.z, x.w += u.w;
      y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
      l += part_l[r][i];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    // positions 4 lane, ...: channels 16 (lane / 4) + 2 (lane % 4), + 8, + 1, + 9
    float* to = &far[r][16 * (lane >> 2) + 2 * (lane & 3)];
    to[0] = x.x * inv;
    to[8] = x.y * inv;
    to[1] = x.z * inv;
    to[9] = x.w * inv;
    reinterpret_cast<float4*>(near[r])[lane] = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
  }
  __syncthreads();
  float out[ROWS];
  times_rotation(f, far, out);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float z = out[i] + near[i][n], next = __shfl_xor_sync(0xffffffffu, z, 2);
    const int row = row0 + i;
    if ((threadIdx.x & 3) == 0 && row < rows)   // outputs n and n + 1
      reinterpret_cast<uint32_t*>(B.out + ((size_t)(A.row[ri] + (row >> A.lg)) * A.Hq + head * G + (row & (G - 1))) * D)[n >> 1] =
          bf16x2(z, next);
  }
}

struct MergeRowsSmem {
  alignas(16) uint16_t r[D][PITCH];            // fp16, columns in unpack_values()'s order
  alignas(16) uint16_t row[8][UNIT][PITCH];    // a warp's rows: the history's sums (fp16), then the results (bf16)
};
// A warp takes 16 rows of one request and kv head at a time; the CTA keeps that head's rotation.  (The history's
// sums, times a power of two of the row's, and R are rounded to fp16, 2^-11 each, an eighth of what the result's
// rounding adds.)
template <bool PAIR>
__global__ void __launch_bounds__(MG_THREADS, 2)
    chunk_merge_rows_kernel(const __grid_constant__ DevCache c, const __grid_constant__ ScanArgs A,
                            const __grid_constant__ MergeArgs B, int per_head) {
  extern __shared__ __align__(16) uint8_t mr_raw[];
  MergeRowsSmem& sm = *reinterpret_cast<MergeRowsSmem*>(mr_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = 1 << A.lg;
  const int head = blockIdx.x / per_head;
  {
    const float* m = c.rot_v + ((size_t)A.layer * c.Hkv + head) * D * D;   // (before the grid's dependency)
#pragma unroll 4
    for (int i = threadIdx.x; i < D * (D / 16); i += MG_THREADS) {
      const int n = i / (D / 16), p = i % (D / 16);
      float f[16];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(f + 4 * j) = reinterpret_cast<const float4*>(m + (size_t)n * D + 16 * p)[j];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint4*>(&sm.r[n][16 * p + 8 * j]) =
            make_uint4(f16x2(f[4 * j], f[4 * j + 8]), f16x2(f[4 * j + 1], f[4 * j + 9]), f16x2(f[4 * j + 2], f[4 * j + 10]),
                       f16x2(f[4 * j + 3], f[4 * j + 11]));
    }
  }
  grid_dep_launch();
  grid_dep_wait();
  __syncthreads();
  constexpr int BLOCK = PAIR ? 2 * SC_ROWS : SC_ROWS;
  constexpr size_t STEP = (size_t)(PAIR ? 2 : 1) * SC_ROWS * PARTIAL_FLOATS;
  const size_t near_step = (size_t)c.Hkv * (2 * SC_ROWS) * PARTIAL_FLOATS;
  uint16_t (*buf)[PITCH] = sm.row[warp];
  for (int unit = blockIdx.x % per_head + per_head * warp; unit < B.chunks; unit += per_head * 8) {
    int ri = 0, hi = A.n;
    while (hi - ri > 1) {
      const int mid = (ri + hi) >> 1;
      if (B.chunk[mid] <= unit) ri = mid; else hi = mid;
    }
    const int row0 = (unit - B.chunk[ri]) * UNIT, last = (A.m[ri] << A.lg) - 1 - row0;   // the unit's last row
    const int64_t each = A.tiles[ri] + A.setup, k = (int64_t)head * A.blocks[ri] + row0 / BLOCK, start = A.cost[ri] + k * each;
    const int64_t c0 = chunk_of(A, start + A.setup), c1 = chunk_of(A, start + each - 1);
    const int count = static_cast<int>(c1 - c0 + 1) * (PAIR ? 1 : 2);
    const float* scan = A.records + ((size_t)(A.segment[ri] + k + c0) * 2 + (PAIR ? row0 % BLOCK / SC_ROWS : 0)) * SC_ROWS * PARTIAL_FLOATS +
                        (size_t)(row0 % SC_ROWS) * PARTIAL_FLOATS;
    const int back = B.near_blocks - 1 - (B.near_start[ri] + row0 / (2 * SC_ROWS));
    const float* bf = B.near + (((size_t)back * B.near_splits * c.Hkv + head) * (2 * SC_ROWS) + row0 % (2 * SC_ROWS)) * PARTIAL_FLOATS;
    // lane r: row r's maximum, weights and their sum (rows behind the last one as that)
    const int mine = min(lane % UNIT, last) * PARTIAL_FLOATS;
    float top = NEG_INF, l = 0.0f;
#pragma unroll 4
    for (int j = 0; j < count; ++j) top = fmaxf(top, scan[j * STEP + mine + PARTIAL_M]);
    for (int j = 0; j < B.near_splits; ++j) top = fmaxf(top, bf[j * near_step + mine + PARTIAL_M]);
    // (a row without a maximum goes the same way: a NaN query's sums are NaN)
    const float ref = top == NEG_INF ? 0.0f : top;
    for (int j = 0; j < B.near_splits; ++j) l = fmaf(bf[j * near_step + mine + PARTIAL_L], ex2f(bf[j * near_step + mine + PARTIAL_M] - ref), l);
#pragma unroll 4
    for (int j = 0; j < count; ++j) l = fmaf(scan[j * STEP + mine + PARTIAL_L], ex2f(scan[j * STEP + mine + PARTIAL_M] - ref), l);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    float down = 1.0f;   // of lane's row: what undoes its power of two
    __syncwarp();
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {   // eight rows, four channels a lane
      float4 sum[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) sum[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int j = 0; j < count; ++j) {
        const float f = ex2f(scan[j * STEP + mine + PARTIAL_M] - ref);
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = reinterpret_cast<const float4*>(scan + j * STEP + min(8 * half + r, last) * PARTIAL_FLOATS)[lane];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float w = __shfl_sync(0xffffffffu, f, 8 * half + r);
          sum[r].x = fmaf(v[r].x, w, sum[r].x);
          sum[r].y = fmaf(v[r].y, w, sum[r].y);
          sum[r].z = fmaf(v[r].z, w, sum[r].z);
          sum[r].w = fmaf(v[r].w, w, sum[r].w);
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float top = fmaxf(fmaxf(fabsf(sum[r].x), fabsf(sum[r].y)), fmaxf(fabsf(sum[r].z), fabsf(sum[r].w)));
        const int e = row_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top))));
        const float up = pow2(e);
        if (lane % UNIT == 8 * half + r) down = pow2(-e) * inv;
        *reinterpret_cast<uint2*>(&buf[8 * half + r][4 * lane]) =
            make_uint2(f16x2(sum[r].x * up, sum[r].y * up), f16x2(sum[r].z * up, sum[r].w * up));
      }
    }
    const float down0 = __shfl_sync(0xffffffffu, down, lane / 4), down1 = __shfl_sync(0xffffffffu, down, lane / 4 + 8);
    __syncwarp();
    uint32_t a[8][4];
#pragma unroll
    for (int s = 0; s < 8; ++s) ldsm4(a[s], smem_u32(&buf[lane & 15][16 * s + 8 * (lane >> 4)]));
    __syncwarp();
    const int r0 = min(lane / 4, last) * PARTIAL_FLOATS, r1 = min(lane / 4 + 8, last) * PARTIAL_FLOATS;
    float x[16][4];
#pragma unroll
    for (int n = 0; n < 16; n += 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] = x[n + 1][i] = 0.0f;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t b[4];
        ldsm4(b, smem_u32(&sm.r[8 * n + (lane & 7) + 8 * (lane >> 4)][16 * s + 8 * ((lane >> 3) & 1)]));
        mma_f16(x[n], a[s][0], a[s][1], a[s][2], a[s][3], b[0], b[1]);
        mma_f16(x[n + 1], a[s][0], a[s][1], a[s][2], a[s][3], b[2], b[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[n][i] *= i < 2 ? down0 : down1, x[n + 1][i] *= i < 2 ? down0 : down1;
    }
    for (int j = 0; j < B.near_splits; ++j) {
      const float f = ex2f(bf[j * near_step + mine + PARTIAL_M] - ref) * inv;
      const float w0 = __shfl_sync(0xffffffffu, f, lane / 4), w1 = __shfl_sync(0xffffffffu, f, lane / 4 + 8);
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const float2 y = *reinterpret_cast<const float2*>(bf + j * near_step + r0 + 8 * n + 2 * (lane & 3));
        const float2 z = *reinterpret_cast<const float2*>(bf + j * near_step + r1 + 8 * n + 2 * (lane & 3));
        x[n][0] = fmaf(y.x, w0, x[n][0]);
        x[n][1] = fmaf(y.y, w0, x[n][1]);
        x[n][2] = fmaf(z.x, w1, x[n][2]);
        x[n][3] = fmaf(z.y, w1, x[n][3]);
      }
    }
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      *reinterpret_cast<uint32_t*>(&buf[lane / 4][8 * n + 2 * (lane & 3)]) = bf16x2(x[n][0], x[n][1]);
      *reinterpret_cast<uint32_t*>(&buf[lane / 4 + 8][8 * n + 2 * (lane & 3)]) = bf16x2(x[n][2], x[n][3]);
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < UNIT / 2; ++u) {
      const int r = 2 * u + lane / 16, rr = row0 + r;
      if (r <= last)
        reinterpret_cast<uint4*>(B.out + ((size_t)(A.row[ri] + (rr >> A.lg)) * A.Hq + head * G + (rr & (G - 1))) * D)[lane % 16] =
            *reinterpret_cast<const uint4*>(&buf[r][8 * (lane % 16)]);
    }
    __syncwarp();
  }
}

// A kernel's shared memory, set once per device (regs: what a split at run time counts on; the build checks it too).
template <typename K>
cudaError_t set_up(K kernel, int bytes, std::atomic<unsigned>& done, int regs = 0) {
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

template <int GK, bool PAIR, bool FEW>
cudaError_t scan(const DevCache& c, const ScanArgs& a, const CUtensorMap& q_map, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(ScanSmem<GK, PAIR>)) + 1024;
  static std::atomic<unsigned> done;
  const cudaError_t e = set_up(chunk_scan_kernel<GK, PAIR, FEW>, bytes, done, SC_REGS);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_scan_kernel<GK, PAIR, FEW>, static_cast<unsigned>(a.ctas), SC_THREADS, bytes, s, c, a, q_map);
}
// CTAs of a kv head, of work for so many warps: two per SM in all.  (Units go to CTAs first, then to their warps: a unit's
// time is its loads', which eight warps of an SM share: 150 tokens over 2K 37.7 us, 48.5 with CTAs filled up.)
int ctas_per_head(int64_t units, int hkv, int sms) {
  const int64_t fair = 2 * sms / hkv > 1 ? 2 * sms / hkv : 1;
  return static_cast<int>(units < fair ? units : fair);
}
void count_chunks(const ScanArgs& a, MergeArgs& b, int rows) {
  b.chunks = 0;
  for (int i = 0; i < a.n; ++i) {
    b.chunk[i] = b.chunks;
    b.chunks += ((a.m[i] << a.lg) + rows - 1) / rows;
  }
}
template <bool PAIR>
cudaError_t merge(const DevCache& c, const ScanArgs& a, MergeArgs& b, int sms, cudaStream_t s) {
  static std::atomic<unsigned> done;
  count_chunks(a, b, UNIT);
  // few rows have many records: two or four rows a CTA spread them
  if ((int64_t)b.chunks * c.Hkv < sms) {
    auto few = [&](auto rows) {
      constexpr int ROWS = decltype(rows)::value;
      count_chunks(a, b, ROWS);
      return launch_dependent(chunk_merge_few_kernel<PAIR, ROWS>, static_cast<unsigned>(b.chunks * c.Hkv), MG_THREADS, 0, s, c, a, b);
    };
    return (int64_t)b.chunks * c.Hkv * (UNIT / 2) <= sms ? few(std::integral_constant<int, 2>()) : few(std::integral_constant<int, FEW>());
  }
  constexpr int bytes = static_cast<int>(sizeof(MergeRowsSmem));
  const cudaError_t e = set_up(chunk_merge_rows_kernel<PAIR>, bytes, done);
  if (e != cudaSuccess) return e;
  const int per_head = ctas_per_head(b.chunks, c.Hkv, sms);
  return launch_dependent(chunk_merge_rows_kernel<PAIR>, static_cast<unsigned>(per_head * c.Hkv), MG_THREADS, bytes, s, c, a,
                          b, per_head);
}

}  // namespace

cudaError_t launch_rotate_queries(const DevCache& c, const RotateArgs& a, int sms, cudaStream_t s) {
  const int64_t few = (((int64_t)a.rows << a.lg) + FEW - 1) / FEW * c.Hkv;
  if (few <= 2 * sms) return launch_dependent(rotate_few_kernel, static_cast<unsigned>(few), MG_THREADS, 0, s, c, a);
  constexpr int bytes = static_cast<int>(sizeof(RotateSmem));
  static std::atomic<unsigned> done;
  const cudaError_t e = set_up(rotate_queries_kernel, bytes, done);
  if (e != cudaSuccess) return e;
  const int per_head = ctas_per_head((((int64_t)a.rows << a.lg) + UNIT - 1) / UNIT, c.Hkv, sms);
  return launch_dependent(rotate_queries_kernel, static_cast<unsigned>(per_head * c.Hkv), MG_THREADS, bytes, s, c, a, per_head);
}
cudaError_t launch_chunk_scan(const DevCache& c, const ScanArgs& a, bool pair, const CUtensorMap& q_map, cudaStream_t s) {
  int rows = 0;
  for (int i = 0; i < a.n; ++i) rows = a.m[i] << a.lg > rows ? a.m[i] << a.lg : rows;
  auto go = [&](auto gk) {
    constexpr int GK = decltype(gk)::value;
    return pair ? scan<GK, true, false>(c, a, q_map, s) : rows > SC_FEW ? scan<GK, false, false>(c, a, q_map, s) : scan<GK, false, true>(c, a, q_map, s);
  };
  return c.gk == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
}
cudaError_t launch_chunk_merge(const DevCache& c, const ScanArgs& a, MergeArgs& b, bool pair, int sms, cudaStream_t s) {
  return pair ? merge<true>(c, a, b, sms, s) : merge<false>(c, a, b, sms, s);
}

}  // namespace oscar
