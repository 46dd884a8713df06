// Windowed attention of many query rows over BF16 pages (prefill), on tcgen05.
//
// A CTA takes 256 query rows of one kv head: two tiles of 128 rows, a row being a
// (token, head of the group) pair, token by token, so the G heads of a group share
// every key and value that is loaded and the causal edge crosses few tiles.  It
// walks the pages that its rows see, two at a time: the sinks' first, then the
// window's.  Per key tile and query tile
//   S = Q K^T            128 x 128 x 128, tcgen05.mma, both operands in shared memory
//   p = exp2(S scale - m)   one thread per row, m the running maximum
//   O = O + P V          tcgen05.mma, P from TMEM, O in TMEM
// The reference m of a row moves only when exceeded by 2^8; then the row's sum and
// its O are scaled (tcgen05.ld / st), otherwise O stays where it is.  P is rounded to
// bf16 for bf16 outputs (each weight off by at most 2^-8, as much as the output's own
// rounding); for fp32 outputs it is carried as three bf16 parts (24 bits).  Sums are taken
// of the unrounded weights, in fp32.
//
// fp32 outputs take one query tile a CTA, and the second's columns keep the tensor core's
// accumulation, which truncates, from showing: the small parts' products go to a sum of
// their own (in O's they would add 16 truncations a key tile to 8), and every four key tiles
// O's sum is added to a total, by fp32 additions (900 queries of 64 heads on 16K keys of 8:
// error 1.1e-6 and 985 to 1012 us, 1.9e-5 and 920 without the total, plain fp32 2.6e-6; the
// floor is 241 us).  P is then handed over 64 keys at a time, in the columns that S leaves.
//
// Roles: warps 0-3 and 4-7 the softmax of query tile 0 and 1, one thread per row (TMEM
// lane = row); warps 8 and 9 the products of query tile 0 and 1; warp 10 the TMA copies;
// warp 11 looks the items up, four ahead (each role doing that for itself took up to 2500
// cycles between two items).
// A query tile's chain is S -> softmax -> PV -> S of the next key tile, since P lies over
// S in TMEM (S0, S1, O0, O1 take all 512 columns); the two query tiles' chains interleave.
// P is handed over in two parts.  Issuing is synchronous (64 cycles a product of
// 128 x 128 x 16, as long as it runs; 110 a commit, 140 a wait even when ready), so one
// warp issuing for both tiles left the tensor core idle for 1100 of 3430 cycles a key
// tile; hence a warp for each, and V of a key tile and K of the next share a stage (two
// stages of 64 KB), one wait and one commit.  The two take turns, [PV, S] of a key tile
// each: left to themselves both tiles fall into step, softmax against softmax and product
// against product (3540 cycles a key tile).
//
// One persistent CTA per SM walks the items (256 rows x kv head), so that the copies and
// the first products of an item run under the end of the one before.  Where the items
// would leave most SMs idle (a few query tokens on a long cache) an item's key tiles are
// split, its unnormalised rows go to the workspace and a second kernel folds them.
//
// Bound by the tensor core: 16K tokens, GQA 4, window 4096: 602 us a call in a loop of
// seconds (1.6 PFLOP/s; at the power cap, SM clock 1657 MHz), 540 us in one of a few ms (1.8
// PFLOP/s), the tensor pipe 80 % busy (a key tile of both query tiles takes 2310 cycles, its
// products 2048).  Ragged, GQA 8, window 1024: 229 us (1927 MHz) and 218 us, 66 %, since a
// quarter of an item's time is its ends.
#include <atomic>

#include "paged_device.cuh"

namespace oscar {
namespace {

using namespace paged;

constexpr int PF_MMA_WARP = 8, PF_TMA_WARP = 10, PF_ITEM_WARP = 11;
constexpr int PF_THREADS = 32 * 12;            // three warpgroups
// Registers a thread: 168 at launch (three warpgroups share 504), then 208 for the
// softmax's two warpgroups, which hold a row of logits each, and 88 for the third.
constexpr int PF_REGS = 168, PF_SOFTMAX_REGS = 208, PF_OTHER_REGS = 88;
static_assert(2 * PF_SOFTMAX_REGS + PF_OTHER_REGS <= 3 * PF_REGS, "a split above the launch's registers waits forever");
constexpr int PF_STAGES = 2;                   // of V of a key tile and K of the next
constexpr int PF_FIRST = 64;                   // keys of P handed over first
constexpr int PF_PARTS = 3;                    // parts of P for fp32 outputs
constexpr int PF_FLUSH = 4;                    // key tiles between additions to the total (fp32 outputs)
constexpr int PF_ITEMS = 4;                    // items looked up ahead
constexpr int PF_READERS = 11;                 // warps that read them
constexpr int PF_ROWS = 128;                   // rows of a query tile
constexpr int PF_KEYS = 2 * PAGE;              // keys of a tile
constexpr int TILE_BYTES = 128 * D * 2;        // a Q, K or V tile

struct PrefillArgs {
  PagedView p;
  AttnArgs a;
  int n, G, lg;                           // lg = log2 G
  int tiles;                              // query tiles of an item, at most
  int splits, items;                      // parts of an item's key tiles; items in all, parts counted
  float* partials;                        // [items][128 tiles][PARTIAL_FLOATS] where splits > 1
  int32_t len[PAGED_MAX_REQ];
  int32_t m[PAGED_MAX_REQ];
  int32_t row[PAGED_MAX_REQ];
  int32_t table[PAGED_MAX_REQ];
  int32_t bstart[PAGED_MAX_REQ + 1];      // blocks of 128 tiles rows before request i (one kv head)
};

// The keys that the rows at positions [pmin, pmax] see, as a list of pages: [0, sink),
// then [first, first + pages - sink).  A key tile is two neighbours of the list, not of
// the cache: four sinks cost a window of 1024 half a tile, not a whole one.
struct KeyTiles {
  int sink, first, pages, count;
  int lo, sinks, pmax;     // tokens t <= pmax with t < sinks or t >= lo are seen by some row
  __device__ static KeyTiles of(int pmin, int pmax, int window, int sinks) {
    KeyTiles k;
    k.pmax = pmax;
    k.sinks = min(sinks, pmax + 1);
    k.lo = window > 0 ? max(0, pmin - window + 1) : pmax + 1;
    k.sink = (k.sinks + PAGE - 1) / PAGE;
    k.first = max(k.lo / PAGE, k.sink);
    const int end = window > 0 ? pmax / PAGE + 1 : 0;
    k.pages = k.sink + max(0, end - k.first);
    k.count = (k.pages + 1) / 2;
    return k;
  }
  // first token of page v of the list; behind its end, tokens that no row sees
  __device__ int base(int v) const { return v >= pages ? PAGED_NO_TOKEN : (v < sink ? v : first + (v - sink)) * PAGE; }
  // whether some row sees token t; all of page v of the list
  __device__ bool any(int t) const { return t <= pmax && (t < sinks || t >= lo); }
  __device__ bool all(int v) const {
    const int t = base(v);
    return t + PAGE - 1 <= pmax && (t + PAGE <= sinks || t >= lo);
  }
};

// One item: up to 256 query rows (128 for fp32 outputs) of a kv head and their key tiles [j0, j1) of kt.
struct alignas(16) Item {
  int index;               // -1: no more items
  int head, table, row;    // kv head, row of the page table, first row of q and out
  int tokens, p0, j0, j1;  // query tokens and the first one's position; key tiles
  KeyTiles kt;
  __device__ int tiles(int per_tile) const { return tokens > per_tile ? 2 : 1; }
  // Item of a CTA's turn.  Later blocks of a request see more keys and come first; every
  // other round goes through the CTAs backwards, so that the longer items of a round fall
  // to different CTAs.
  __device__ void load(const PrefillArgs& A, int turn) {
    const int grid = gridDim.x, at = turn & 1 ? grid - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x);
    index = turn * grid + at;
    if (index >= A.items) {
      index = -1;
      return;
    }
    head = index % A.p.Hkv;
    const int rest = index / A.p.Hkv, split = rest % A.splits, blk = A.bstart[A.n] - 1 - rest / A.splits;
    int hi = A.n, ri = 0;
    while (hi - ri > 1) {
      const int mid = (ri + hi) >> 1;
      if (A.bstart[mid] <= blk) ri = mid; else hi = mid;
    }
    const int m = A.m[ri], per_tile = PF_ROWS >> A.lg;
    const int tok0 = (blk - A.bstart[ri]) * A.tiles * per_tile;   // first token of the block, of the request's m
    table = A.table[ri];
    row = A.row[ri] + tok0;
    tokens = min(A.tiles * per_tile, m - tok0);
    p0 = A.len[ri] - m + tok0;
    kt = KeyTiles::of(p0, p0 + tokens - 1, A.a.window, A.a.sinks);
    j0 = kt.count * split / A.splits;
    j1 = kt.count * (split + 1) / A.splits;
  }
};

struct alignas(1024) PrefillSmem {
  alignas(1024) uint8_t q[2][TILE_BYTES];      // per tile: two halves of 64 channels, [128 rows][128 B] swizzled
  alignas(1024) uint8_t kv[PF_STAGES][2][TILE_BYTES];   // V of key tile j - 1, K of key tile j
  alignas(16) uint8_t out[8][32 * 128];                 // per softmax warp: 128 bytes of its 32 rows
  uint64_t q_full[2], q_empty[2], kv_full[PF_STAGES], kv_empty[PF_STAGES];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_empty[2];   // per query tile (and half of the keys)
  uint64_t p_empty;                              // the first half's products are done (fp32 outputs)
  uint64_t turn[2];                              // the other tile's products of a key tile are issued
  uint64_t item_full[PF_ITEMS], item_empty[PF_ITEMS];
  Item item[PF_ITEMS];
  uint32_t tmem;
};
static_assert(sizeof(PrefillSmem) + 1024 <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

#define OSCAR_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define OSCAR_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of the warp's lanes
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : OSCAR_R8(r, 0), OSCAR_R8(r, 8), OSCAR_R8(r, 16), OSCAR_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : OSCAR_R8(r, 0), OSCAR_R8(r, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      OSCAR_W8(r, 0), OSCAR_W8(r, 8)
      : "memory");
}
#undef OSCAR_R8
#undef OSCAR_W8

// Shared-memory descriptors with the 128-byte swizzle.  K-major (Q, K): rows of 128 B,
// groups of 8 rows 1024 B apart.  N-major (V): groups of 8 keys 1024 B apart, the
// second 64 channels 16 KB on.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_nmajor(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(16384 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, bf16 operands, fp32 result, M = N = 128; PV has its B operand N-major.
constexpr uint32_t IDESC_QK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t IDESC_PV = IDESC_QK | (1u << 16);

// Issued by one elected lane of a converged warp: the code around stays uniform, so that
// descriptors are computed in uniform registers (under an if of one lane, each product
// cost its six operand moves, and a key tile of the issuing warp 4700 cycles).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_elected(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}

// A warp's wait (skipped where an earlier one gave up), the same answer for all lanes.
// All lanes poll: handing one lane's answer round took 200 cycles more.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, bool ok) {
  return ok && __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

template <bool F32, bool SPLIT>
__global__ void __launch_bounds__(PF_THREADS, 1)
    paged_prefill_kernel(const __grid_constant__ PrefillArgs A, const __grid_constant__ CUtensorMap q_map,
                         const __grid_constant__ CUtensorMap kv_map) {
  extern __shared__ uint8_t pf_raw[];
  PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(pf_raw + (-smem_u32(pf_raw) & 1023u));
  // (through a shuffle: uniform for the compiler too)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < PF_STAGES; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 2);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.q_full[a], 1);
      mbar_init(&sm.q_empty[a], 1);
      mbar_init(&sm.s_full[a], 1);
      mbar_init(&sm.o_empty[a], 4);
      mbar_init(&sm.p_full[a][0], 4);
      mbar_init(&sm.p_full[a][1], 4);
      mbar_init(&sm.o_full[a], 1);
      mbar_init(&sm.turn[a], 1);
    }
    for (int s = 0; s < PF_ITEMS; ++s) {
      mbar_init(&sm.item_full[s], 1);
      mbar_init(&sm.item_empty[s], PF_READERS);
    }
    mbar_init(&sm.p_empty, 1);
    mbar_init_fence();
    prefetch_map(&q_map);
    prefetch_map(&kv_map);
  }
  if (warp == PF_MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  grid_dep_launch();
  grid_dep_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;   // all 512 columns are the CTA's
  auto gave_up = [&]() {
    if (A.p.err) atomicOr(A.p.err, PAGED_ERR_TIMEOUT);
  };

  const int per_tile = PF_ROWS >> A.lg;
  if (warp >= PF_MMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PF_OTHER_REGS));
    if (warp == PF_ITEM_WARP) {
      // ---- items
      if (lane == 0) {
        for (int turn = 0;; ++turn) {
          const int at = turn % PF_ITEMS;
          if (turn >= PF_ITEMS && !mbar_wait(&sm.item_empty[at], (turn / PF_ITEMS - 1) & 1)) {
            gave_up();
            break;
          }
          Item next;
          next.load(A, turn);
          sm.item[at] = next;
          mbar_arrive(&sm.item_full[at]);
          if (next.index < 0) break;
        }
      }
    } else if (warp == PF_TMA_WARP) {
      // ---- copies
      if (lane == 0) {
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity); };
        int stage = 0, q_loads[2] = {0, 0};   // stages and query tiles loaded so far
        for (int turn = 0; ok; ++turn) {
          const int at = turn % PF_ITEMS;
          wait(&sm.item_full[at], (turn / PF_ITEMS) & 1);
          if (!ok) break;
          const Item it = sm.item[at];
          mbar_arrive(&sm.item_empty[at]);
          if (it.index < 0) break;
          const KeyTiles& kt = it.kt;
          if (it.j0 == it.j1) continue;
          const int tiles = it.tiles(per_tile);
          for (int a = 0; a < tiles; ++a) {
            if (q_loads[a] > 0) wait(&sm.q_empty[a], (q_loads[a] - 1) & 1);
            if (!ok) break;
            ++q_loads[a];
            mbar_expect_tx(&sm.q_full[a], TILE_BYTES);
            for (int h = 0; h < 2; ++h)
              tma_load_3d(sm.q[a] + h * (TILE_BYTES / 2), &q_map, 64 * h, it.head * A.G,
                          it.row + a * per_tile, &sm.q_full[a]);
          }
          const int32_t* pt = A.p.table + (size_t)it.table * A.p.max_pages;
          // records of the pages of key tile j, -1: no second one
          auto tile_records = [&](int j, int (&rec)[2]) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              rec[u] = -1;
              if (2 * j + u >= kt.pages) continue;
              int page = pt[kt.base(2 * j + u) / PAGE];
              if (page < 0 || page >= A.p.num_pages) {
                if (A.p.err) atomicOr(A.p.err, PAGED_ERR_PAGE);
                page = 0;
              }
              rec[u] = static_cast<int>(2 * ((int64_t)page * A.p.Hkv + it.head));
            }
          };
          auto load = [&](uint8_t* dst, const int (&rec)[2], int which, uint64_t* bar) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (rec[u] >= 0)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  tma_load_3d(dst + h * (TILE_BYTES / 2) + u * (TILE_BYTES / 4), &kv_map, 64 * h, 0, rec[u] + which, bar);
          };
          int prev[2] = {-1, -1}, cur[2];
          tile_records(it.j0, cur);
          for (int j = it.j0; j <= it.j1 && ok; ++j, ++stage) {   // V of tile j - 1, K of tile j
            const int st = stage % PF_STAGES;
            if (stage >= PF_STAGES) wait(&sm.kv_empty[st], (stage / PF_STAGES - 1) & 1);
            if (!ok) break;
            const int pages = (prev[0] >= 0) + (prev[1] >= 0) + (cur[0] >= 0) + (cur[1] >= 0);
            mbar_expect_tx(&sm.kv_full[st], pages * (TILE_BYTES / 2));
            load(sm.kv[st][0], prev, 1, &sm.kv_full[st]);
            load(sm.kv[st][1], cur, 0, &sm.kv_full[st]);
            prev[0] = cur[0], prev[1] = cur[1];
            cur[0] = cur[1] = -1;
            if (j + 1 < it.j1) tile_records(j + 1, cur);
          }
        }
        if (!ok) gave_up();
        // nothing may arrive after the CTA: copies in flight, and the last commits
        for (int k = max(0, stage - PF_STAGES); k < stage; ++k) {
          mbar_wait(&sm.kv_full[k % PF_STAGES], (k / PF_STAGES) & 1);
          if (ok) mbar_wait(&sm.kv_empty[k % PF_STAGES], (k / PF_STAGES) & 1);
        }
        for (int a = 0; a < 2; ++a)
          if (q_loads[a] > 0) {
            mbar_wait(&sm.q_full[a], (q_loads[a] - 1) & 1);
            if (ok) mbar_wait(&sm.q_empty[a], (q_loads[a] - 1) & 1);
          }
      }
    } else if (warp < PF_TMA_WARP) {
      // ---- products of query tile a
      const int a = warp - PF_MMA_WARP;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { ok = mbar_wait_warp(bar, parity, ok); };
      const uint64_t q = desc_kmajor(smem_u32(sm.q[a])), k_desc = desc_kmajor(smem_u32(sm.kv[0][1])),
                     v_desc = desc_nmajor(smem_u32(sm.kv[0][0]));
      const uint32_t s_col = 128 * a, o_col = 256 + 128 * a;
      int stage = 0;      // stages taken so far
      int batch = 0;      // [PV, S] turns of items with two tiles
      int tile = 0;       // key tiles of this query tile
      int done = 0;       // items of this query tile
      for (int turn = 0; ok; ++turn) {
        const int at = turn % PF_ITEMS;
        wait(&sm.item_full[at], (turn / PF_ITEMS) & 1);
        if (!ok) break;
        const Item it = sm.item[at];
        __syncwarp();
        mbar_arrive_elected(&sm.item_empty[at]);
        if (it.index < 0) break;
        const KeyTiles& kt = it.kt;
        if (it.j0 == it.j1) continue;
        const bool two = it.tiles(per_tile) == 2;
        if (a > 0 && !two) {   // no rows: only free the stages
          for (int j = it.j0; j <= it.j1 && ok; ++j, ++stage) {
            wait(&sm.kv_full[stage % PF_STAGES], (stage / PF_STAGES) & 1);
            if (ok) mbar_arrive_elected(&sm.kv_empty[stage % PF_STAGES]);
          }
          continue;
        }
        auto pass_turn = [&]() {
          if (two) mbar_arrive_elected(&sm.turn[a ^ 1]);
        };
        auto score = [&](int st, bool pass) {
          const uint64_t k = k_desc + st * (2 * TILE_BYTES >> 4);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if (s == 6 && pass) pass_turn();   // the last two cover the other warp's waking
            const uint64_t off = ((s >> 2) * (TILE_BYTES / 2) + (s & 3) * 32) >> 4;
            mma_ss(s_col, q + off, k + off, IDESC_QK, s > 0);
          }
          mma_commit(&sm.s_full[a]);
        };
        wait(&sm.q_full[a], done & 1);
        wait(&sm.kv_full[stage % PF_STAGES], (stage / PF_STAGES) & 1);
        if (!ok) break;
        tc_fence_after();
        score(stage % PF_STAGES, false);
        mma_commit(&sm.kv_empty[stage % PF_STAGES]);
        ++stage;
        if (done > 0) wait(&sm.o_empty[a], (done - 1) & 1);   // the last item's rows are out of O
        for (int j = it.j0; j < it.j1 && ok; ++j, ++stage, ++tile, batch += two) {
          const int st = stage % PF_STAGES;
          wait(&sm.kv_full[st], (stage / PF_STAGES) & 1);
          if (!kt.all(2 * j) || !kt.all(2 * j + 1)) {
            // value rows that no row sees may hold anything (or were not copied): zero them
            // (both tiles' warps do, each before its own product)
            uint8_t* v = sm.kv[st][0];
            for (int r = lane >> 3; r < PF_KEYS; r += 4)
              if (!kt.any(kt.base(2 * j + r / PAGE) + r % PAGE)) {
                uint4* dst = reinterpret_cast<uint4*>(v + r * 128 + (lane & 7) * 16);
                dst[0] = make_uint4(0, 0, 0, 0);
                dst[TILE_BYTES / 32] = make_uint4(0, 0, 0, 0);
              }
            fence_async_smem();
            __syncwarp();
          }
          const uint64_t v = v_desc + st * (2 * TILE_BYTES >> 4);
          if (two && a + batch > 0) wait(&sm.turn[a], (a == 0 ? batch - 1 : batch) & 1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // P's parts
            wait(&sm.p_full[a][h], tile & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int s = h ? PF_FIRST / 16 : 0; s < (h ? 8 : PF_FIRST / 16); ++s) {   // 16 keys
              const uint32_t col = s_col + (F32 ? 0 : 64 * (s / 4)) + 8 * (s % 4);
              const bool first = s == 0 && (F32 ? (j - it.j0) % PF_FLUSH == 0 : j == it.j0);
#pragma unroll
              for (int part = 0; part < (F32 ? PF_PARTS : 1); ++part)
                mma_ts(o_col + (part ? 128 : 0), col + 32 * part, v + (2048 * s >> 4), IDESC_PV,
                       (part == 0 ? !first : j > it.j0 || s > 0 || part > 1) ? 1u : 0u);
            }
            if (F32 && h == 0) mma_commit(&sm.p_empty);
          }
          if (!ok) break;
          if (j + 1 < it.j1) {
            score(st, true);
            if (j + 2 == it.j1) mma_commit(&sm.q_empty[a]);
          } else {
            pass_turn();
            mma_commit(&sm.o_full[a]);
            if (it.j0 + 1 == it.j1) mma_commit(&sm.q_empty[a]);   // the one tile's S was the first
          }
          mma_commit(&sm.kv_empty[st]);
        }
        ++done;
      }
      if (!ok && lane == 0) gave_up();
    }
  } else {
    // ---- softmax of query tile a, one thread per row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PF_SOFTMAX_REGS));
    const int a = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lane_off + 128 * a, to = tmem + lane_off + 256 + 128 * a;
    const float scale2 = A.a.scale2;
    const int tok = a * per_tile + (r >> A.lg);
    bool ok = true;
    int tile = 0, done = 0;   // key tiles and items so far
    for (int turn = 0; ok; ++turn) {
      const int at = turn % PF_ITEMS;
      ok = mbar_wait_warp(&sm.item_full[at], (turn / PF_ITEMS) & 1, ok);
      if (!ok) break;
      const Item& it = sm.item[at];
      auto release = [&]() {   // the warp has read the item
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.item_empty[at]);
      };
      if (it.index < 0) break;
      if (a >= it.tiles(per_tile)) {
        release();
        continue;
      }
      const int pmin = it.p0 + a * per_tile, pmax = it.p0 + min(it.tokens, (a + 1) * per_tile) - 1;
      const int pos = min(it.p0 + tok, pmax);
      // pages from t0 that every row sees whole: t0 <= all_to and (t0 <= all_sinks or t0 > all_from)
      const int all_to = pmin - (PAGE - 1), all_sinks = A.a.sinks - PAGE, all_from = pmax - A.a.window;
      const int lo0 = pos - A.a.window + 1;
      const int sink = it.kt.sink, skip = it.kt.first - it.kt.sink, pages = it.kt.pages, j0 = it.j0, j1 = it.j1;
      float mx = NEG_INF, l = 0.0f;
      for (int j = j0; j < j1; ++j, ++tile) {
        ok = mbar_wait_warp(&sm.s_full[a], tile & 1, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t xr[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, xr + 32 * c);
        tc_wait_ld();
        float* x = reinterpret_cast<float*>(xr);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int v = 2 * j + u, t0 = v >= pages ? PAGED_NO_TOKEN : (v < sink ? v : v + skip) * PAGE;
          if (!(t0 <= all_to && (t0 <= all_sinks || t0 > all_from))) {
            // (bits first: comparing every key took 1500 cycles a page)
            const uint64_t see = visible_bits(pos - t0, lo0 - t0, A.a.sinks - t0);
            const uint32_t half[2] = {static_cast<uint32_t>(see), static_cast<uint32_t>(see >> 32)};
#pragma unroll
            for (int i = 0; i < PAGE; ++i)
              x[PAGE * u + i] = half[i / 32] & (1u << (i % 32)) ? x[PAGE * u + i] : NEG_INF;
          }
        }
        float t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = x[k];
#pragma unroll
        for (int i = 4; i < 124; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) t[k] = max3(t[k], x[i + 2 * k], x[i + 2 * k + 1]);
        const float top = fmaxf(max3(t[0], t[1], max3(t[2], t[3], x[124])), max3(x[125], x[126], x[127])) * scale2;
        const bool raise = top > mx + LAZY_MAX || (mx == NEG_INF && top > NEG_INF);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? (mx == NEG_INF ? 0.0f : ex2f(mx - top)) : 1.0f;
          l *= f;
          if (raise) mx = top;
          if (j > j0) {   // the product before S is done: S was issued after it
#pragma unroll 1
            for (int c = F32 ? -128 : 0; c < (F32 ? 256 : 128); c += 16) {   // in small pieces: the logits are live
              uint32_t o[16];
              tmem_ld16(to + c, o);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(to + c, o);
            }
          }
        }
        if (F32 && j > j0 && (j - j0) % PF_FLUSH == 0) {   // O's sum so far to the total
          tc_wait_st();
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16], total[16];
            tmem_ld16(to + c, o);
            if (j - j0 > PF_FLUSH) {
              tmem_ld16(to - 128 + c, total);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(total[i]));
            }
            tc_wait_ld();
            tmem_st16(to - 128 + c, o);
          }
        }
        const float ref = mx == NEG_INF ? 0.0f : -mx;
        const float2 scale_2 = make_float2(scale2, scale2), ref_2 = make_float2(ref, ref);
        float2 sum[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = make_float2(0.0f, 0.0f);
        // 32 keys at a time: the product of the first part starts while the last is computed
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float2 y[16];
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            y[i] = fma2(make_float2(x[32 * c + 2 * i], x[32 * c + 2 * i + 1]), scale_2, ref_2);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            y[i].x = ex2f(y[i].x);
            y[i].y = ex2f(y[i].y);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            pk[i] = bf16x2(y[i].x, y[i].y);
            sum[i & 3] = add2(sum[i & 3], y[i]);
          }
          // P lies over S, 64 keys in 32 columns (and their other parts in the next ones)
          const int col = (F32 ? 0 : 64 * (c / 2)) + 16 * (c % 2);
          if (F32 && c == 2) {   // the second half lies where the first was
            ok = mbar_wait_warp(&sm.p_empty, tile & 1, ok);
            tc_fence_after();
          }
          tmem_st16(ts + col, pk);
          if constexpr (F32) {
#pragma unroll
            for (int part = 1; part < PF_PARTS; ++part) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                y[i].x -= __uint_as_float(pk[i] << 16);
                y[i].y -= __uint_as_float(pk[i] & 0xffff0000u);
                pk[i] = bf16x2(y[i].x, y[i].y);
              }
              tmem_st16(ts + col + 32 * part, pk);
            }
          }
          if (c == PF_FIRST / 32 - 1 || c == 3) {
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[a][c == 3]);
          }
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
      }
      const bool some = j1 > j0;
      const int tokens = it.tokens;
      const size_t row0 = (size_t)it.row * A.a.Hq + (size_t)it.head * A.G;   // of token 0, head 0 of the group
      float* part = A.partials + ((size_t)it.index * A.tiles * PF_ROWS + a * PF_ROWS) * PARTIAL_FLOATS;
      release();
      if (some) ok = mbar_wait_warp(&sm.o_full[a], done & 1, ok);
      if (!ok) break;
      tc_fence_after();
      const float inv = SPLIT ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
      if constexpr (SPLIT) {
        part[r * PARTIAL_FLOATS + PARTIAL_M] = mx;
        part[r * PARTIAL_FLOATS + PARTIAL_L] = l;
      } else if (tok < tokens && A.a.lse) {
        A.a.lse[row0 + (size_t)tok * A.a.Hq + (r & (A.G - 1))] =
            l != 0.0f ? (mx + log2f(l)) * 0.6931471805599453f : NEG_INF;
      }
      // O's rows, 128 bytes at a time, turned through shared memory so that eight lanes
      // store a row's piece together: a store of one row per lane touches 32 lines, and
      // those of a tile held up the load-store unit for 5500 cycles
      constexpr bool WIDE = F32 || SPLIT;   // fp32 rows: four pieces of 32 channels, else two of 64
      constexpr int PIECE = WIDE ? 32 : 64, SIZE = WIDE ? 4 : 2;
      char* out = SPLIT ? reinterpret_cast<char*>(part)
                        : static_cast<char*>(A.a.out) + (row0 + (size_t)a * per_tile * A.a.Hq) * (D * SIZE);
      const int left = tokens - a * per_tile;   // the tile's tokens
      uint8_t* stage = sm.out[warp];
#pragma unroll 1
      for (int c = 0; c < 128; c += PIECE) {
        uint32_t w[32];
        if (some) {
          uint32_t o[PIECE];
          tmem_ld32(to + c, o);
          if constexpr (!WIDE) tmem_ld32(to + c + 32, o + 32);
          if constexpr (F32) tmem_ld32(to + 128 + c, w);   // the small parts' sum
          tc_wait_ld();
          if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(w[i]));
            if (j1 - j0 > PF_FLUSH) {   // the total
              tmem_ld32(to - 128 + c, w);
              tc_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(w[i]));
            }
          }
          if (c + PIECE == 128) {   // O is read: the next item may write it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_empty[a]);
          }
          if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              w[i] = bf16x2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
          }
        }
        if (!some || l == 0.0f) {
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < 8; ++k) {
          const int rw = 4 * k + lane / 8, rr = 32 * (warp & 3) + rw, tk = rr >> A.lg;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + rw * 128 + (((lane & 7) ^ (rw & 7)) << 4));
          const int at_row = SPLIT ? rr * PARTIAL_FLOATS * SIZE : (tk * A.a.Hq + (rr & (A.G - 1))) * (D * SIZE);
          if (SPLIT || tk < left) *reinterpret_cast<uint4*>(out + at_row + c * SIZE + 16 * (lane & 7)) = v;
        }
        __syncwarp();
      }
      done += some;
    }
    if (!ok && lane == 0) gave_up();
  }
  __syncwarp();
  __syncthreads();
  if (warp == PF_MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Fold the parts of split items: one warp per query row of (token, head).
constexpr int FOLD_WARPS = 8;
__global__ void __launch_bounds__(32 * FOLD_WARPS)
    paged_prefill_fold_kernel(const __grid_constant__ PrefillArgs A) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * FOLD_WARPS + (threadIdx.x >> 5);   // ((block, head), row of the block)
  const int rows = A.tiles * PF_ROWS, r = unit % rows, bh = unit / rows, head = bh % A.p.Hkv, back = bh / A.p.Hkv;
  const int blk = A.bstart[A.n] - 1 - back;
  if (blk < 0) return;
  int ri = 0, hi = A.n;
  while (hi - ri > 1) {
    const int mid = (ri + hi) >> 1;
    if (A.bstart[mid] <= blk) ri = mid; else hi = mid;
  }
  const int tok = (blk - A.bstart[ri]) * (rows >> A.lg) + (r >> A.lg);
  if (tok >= A.m[ri]) return;
  grid_dep_launch();
  grid_dep_wait();
  // part s of the item is at item ((back splits + s) Hkv + head)
  auto at = [&](int s) {
    return A.partials + (((size_t)(back * A.splits + s) * A.p.Hkv + head) * rows + r) * PARTIAL_FLOATS;
  };
  float m = NEG_INF, l = 0.0f;
  for (int s = 0; s < A.splits; ++s) m = fmaxf(m, at(s)[PARTIAL_M]);
  // (a row without a maximum goes the same way: a NaN query's sums are NaN)
  const float ref = m == NEG_INF ? 0.0f : m;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < A.splits; ++s) {
    const float* p = at(s);
    const float f = ex2f(p[PARTIAL_M] - ref);
    const float4 v = reinterpret_cast<const float4*>(p)[lane];
    l = fmaf(p[PARTIAL_L], f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  const size_t row = (size_t)(A.row[ri] + tok) * A.a.Hq + (size_t)head * A.G + (r & (A.G - 1));
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  if (A.a.f32)
    reinterpret_cast<float4*>(static_cast<float*>(A.a.out) + row * D)[lane] = o;
  else
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.a.out) + row * D)[lane] =
        make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
  if (A.a.lse && lane == 0) A.a.lse[row] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : NEG_INF;
}

int item_rows(bool f32) { return f32 ? PF_ROWS : 2 * PF_ROWS; }

}  // namespace

// Parts of an item's key tiles, whatever the lengths: as many as fill the SMs once,
// where the items alone fill less than half of them.
int paged_prefill_splits(int64_t blocks, int hkv, int sms) {
  const int64_t items = blocks * hkv;
  return items == 0 || 2 * items > sms ? 1 : static_cast<int>(sms / items < 32 ? sms / items : 32);
}
int64_t paged_prefill_blocks(int m, int G, bool f32) {
  return ((int64_t)m * G + item_rows(f32) - 1) / item_rows(f32);
}
size_t paged_prefill_partial_bytes(int64_t blocks, int hkv, int sms, bool f32) {
  const int splits = paged_prefill_splits(blocks, hkv, sms);
  return splits == 1 ? 0 : (size_t)blocks * hkv * splits * item_rows(f32) * PARTIAL_FLOATS * sizeof(float);
}

cudaError_t launch_paged_prefill(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a,
                                 const CUtensorMap& q_map, const CUtensorMap& kv_map, void* partials, int sms,
                                 cudaStream_t s) {
  PrefillArgs A;
  A.p = p;
  A.a = a;
  A.n = n;
  A.G = a.Hq / p.Hkv;
  A.lg = A.G == 1 ? 0 : A.G == 2 ? 1 : A.G == 4 ? 2 : 3;
  const int rows = item_rows(a.f32);
  A.tiles = rows / PF_ROWS;
  int64_t blocks = 0, longest = 0;   // longest: key tiles of an item, at most
  for (int i = 0; i < n; ++i) {
    A.len[i] = reqs[i].len;
    A.m[i] = reqs[i].m;
    A.row[i] = reqs[i].row;
    A.table[i] = reqs[i].table;
    A.bstart[i] = static_cast<int32_t>(blocks);
    blocks += paged_prefill_blocks(reqs[i].m, A.G, a.f32);
    const int64_t most = (int64_t)a.window + a.sinks + rows, seen = most < reqs[i].len ? most : reqs[i].len;
    longest = seen / PF_KEYS + 1 > longest ? seen / PF_KEYS + 1 : longest;
  }
  A.bstart[n] = static_cast<int32_t>(blocks);
  const int most = paged_prefill_splits(blocks, p.Hkv, sms);
  // a part has four key tiles or more
  A.splits = static_cast<int>(longest / 4 < most ? (longest / 4 > 1 ? longest / 4 : 1) : most);
  A.partials = static_cast<float*>(partials);
  if (blocks * p.Hkv * A.splits > INT32_MAX / 2) return cudaErrorInvalidValue;
  A.items = static_cast<int>(blocks * p.Hkv * A.splits);
  constexpr int bytes = static_cast<int>(sizeof(PrefillSmem)) + 1024;
  const int which = (a.f32 ? 1 : 0) + (A.splits > 1 ? 2 : 0);
  auto kernel = which == 0   ? paged_prefill_kernel<false, false>
                : which == 1 ? paged_prefill_kernel<true, false>
                : which == 2 ? paged_prefill_kernel<false, true>
                             : paged_prefill_kernel<true, true>;
  static std::atomic<unsigned> done[4];   // devices that have been set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(done[which].load() & (1u << dev))) {
    cudaFuncAttributes attr;   // the registers that the split counts on (the build checks them too)
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != PF_REGS) return cudaErrorInvalidKernelImage;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 32) done[which].fetch_or(1u << dev);
  }
  e = launch_dependent(kernel, A.items < sms ? A.items : sms, PF_THREADS, bytes, s, A, q_map, kv_map);
  if (e != cudaSuccess || A.splits == 1) return e;
  const int64_t warps = blocks * p.Hkv * rows;
  return launch_dependent(paged_prefill_fold_kernel, static_cast<unsigned>((warps + FOLD_WARPS - 1) / FOLD_WARPS),
                          32 * FOLD_WARPS, 0, s, A);
}

}  // namespace oscar
