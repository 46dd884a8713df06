// Attention of a few query rows per request over a paged cache, BF16 or 4-bit:
// the decode form of the windowed attention, and speculative steps of a few
// tokens.
//
//   o_r = sum_t p_rt v_t / sum_t p_rt,  p_rt = exp(scale q_r . k_t)
// over the tokens t <= p_r that the row sees: t < sinks or t > p_r - window.  The
// rows of one (request, kv head) -- its m query tokens times the G heads of the
// group, up to 16 -- share one pass over the keys and values ("segment").
//
// Traffic bounds it (512 B per token and kv head in BF16, 136 or 144 B in 4 bits,
// for 2 x 2 x 128 flops per row), so the split serves the copies alone.  One
// persistent CTA per SM takes an equal contiguous share of all the segments'
// visible units (16 tokens of a BF16 page, a page in 4 bits; units that no row
// sees are not in the list, and pages that hold none are never touched).  Each
// warp streams its own units through its own TMA ring, the copies running on
// across segment borders, and keeps a running (max, sum, o); a segment's warps
// are folded in shared memory, its CTAs by the last of them to finish.
//
// Both contractions run on warp-level mma.sync m16n8k16 with tokens, then channels,
// as the 16 rows: at 4 to 16 query rows the fixed 128-row tile of the tcgen05 MMA
// would be mostly padding, and the products take a tenth of the copies' time.
//  * BF16: q and v are bf16 already; p is carried as three bf16 parts (24 bits), so
//    every product is exact in fp32.
//  * 4 bits: a code c is or-ed into the fp16 number 1024 (or 1024 + 16 c) and one
//    half2 fma makes it c - 8, exact and centred: sums of the positive codes
//    themselves would lose the mean of many values to their common offset and to the
//    matrix unit's one-sided truncation (2.4e-5 of the output at 30K tokens; codes
//    used in place as fp16 subnormals, one operation less, lost the same to the
//    unit's alignment).  q is exact in fp16 after scaling by a power of two (bf16 has
//    8 bits); p s is carried as two fp16 parts (22 bits), scaled by a running power
//    of two that keeps it inside fp16's range:
//      logit = s (q . (c - 8)) + (z + 8 s) sum(q),
//      sum p v = sum (p s) (c - 8) + sum p (z + 8 s).
// The probabilities come out of the first product with a lane holding two tokens
// of a row; movmatrix turns them into the second product's operand.
//
// Measured, GQA 4 unless noted: BF16, 32 requests with an 8K window 165 us (0.98 of the
// copy's rate), one of 100K 67 us (0.92), 16 rows (GQA 8, two query tokens) 20 of 60K 712 us
// (the copy's rate), the smallest call 6 us.  4 bits, 32 of 16K to 64K 238 us (0.90; 59 % of
// the issue slots, 1080 instructions a page), 316 us at 8 rows and 551 us at 16; one of 100K
// at GQA 8 and group 64 35 us, of 30K 14 us: instructions and latency, neither the issue
// slots nor DRAM full, and 6 us to start and to fold.
#include <atomic>

#include "paged_device.cuh"

namespace oscar {
namespace {

using namespace paged;

template <int GK>
struct Format {
  static constexpr int UT = GK == 0 ? 16 : PAGE;                      // tokens per unit
  static constexpr int BYTES = GK == 0 ? UT * 4 * D : i4_record(GK);  // bytes of one unit
};

template <int GK, int NR>
struct DecodeShape {
  // Warps: the BF16 unit is a few instructions for 8 KB, so eight warps keep the
  // copies going; the 4-bit unit is bound by its instructions, so as many warps as the
  // registers and two pages each in shared memory allow.
  static constexpr int NW = GK == 0 || NR == 16 ? 8 : 12;
  static constexpr int THREADS = 32 * NW;
  static constexpr int FOLD = NR == 4 ? 2 : 1;   // warps folded at a time between segments
  static constexpr size_t LIMIT = 232448 - 1024;   // shared memory of a CTA, less the alignment
  static constexpr size_t FIXED = sizeof(float) * FOLD * NR * PARTIAL_FLOATS + 2048 * ((NR + 7) / 8) + 1024;
  static constexpr int FIT = static_cast<int>((LIMIT - FIXED) / (NW * Format<GK>::BYTES));
  static constexpr int STAGES = FIT > 3 ? 3 : FIT;
  static_assert(STAGES >= 2, "a ring needs two stages");
  static_assert(NW <= INT32_MAX - DECODE_MAX_UNITS, "a step past the last unit is an int");
};

template <int GK, int NR>
struct alignas(1024) DecodeSmem {
  static constexpr int STAGES = DecodeShape<GK, NR>::STAGES, NW = DecodeShape<GK, NR>::NW;
  static constexpr int FOLD = DecodeShape<GK, NR>::FOLD;
  alignas(1024) uint8_t ring[NW][STAGES][Format<GK>::BYTES];
  alignas(16) float state[FOLD][NR][PARTIAL_FLOATS];
  alignas(16) uint32_t q[(NR + 7) / 8][8][4][16];   // the first product's B operand: [tile][column][lane % 4][register]
  float q_scale[NR], q_sum[2][NR];
  uint64_t full[NW][STAGES];
  int last;
};

// The visible units of a request: [0, sink) and [first, first + units - sink).  An
// empty list still counts as one unit, so that some CTA writes the zero rows.
struct Units {
  int32_t sink, first, units;
  static Units of(int len, int m, int window, int sinks, int ut) {
    const int64_t lo64 = (int64_t)len - m - window + 1;
    const int lo = lo64 > 0 ? static_cast<int>(lo64) : 0;
    Units u;
    u.sink = ((sinks < len ? sinks : len) + ut - 1) / ut;
    const int end = (len + ut - 1) / ut;
    u.first = lo / ut > u.sink ? lo / ut : u.sink;
    // window 0: only the sinks are seen
    u.units = u.sink + (window > 0 && end > u.first ? end - u.first : 0);
    return u;
  }
  __host__ __device__ int unit(int v) const { return v < sink ? v : first + (v - sink); }
};

struct DecodeArgs {
  PagedView p;
  AttnArgs a;
  int n, m, G, ncta;
  int32_t total;                            // units of the call
  float* partials;
  int32_t* counters;
  // request i; side by side, since each line of the arguments comes from a cold cache
  struct Req {
    int32_t len, row, table;
    int32_t ustart;                         // units before it (all its kv heads)
    Units un;
  } req[PAGED_MAX_REQ];
};

// Position of a CTA's walk over the units u of the call.
struct Cursor {
  int req, head, base, seg_end;   // current segment: units [base, seg_end)
  Units un;
};
template <int UT>
__device__ __forceinline__ void cursor_load(const DecodeArgs& A, Cursor& c) {
  c.un = A.req[c.req].un;
  c.seg_end = c.base + max(c.un.units, 1);
}
template <int UT>
__device__ __forceinline__ void cursor_first(const DecodeArgs& A, Cursor& c, int u) {
  int lo = 0, hi = A.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (A.req[mid].ustart <= u) lo = mid; else hi = mid;
  }
  c.req = lo;
  c.base = A.req[lo].ustart;
  cursor_load<UT>(A, c);
  const int per = c.seg_end - c.base;
  c.head = (u - c.base) / per;
  c.base += c.head * per;
  c.seg_end = c.base + per;
}
template <int UT>
__device__ __forceinline__ void cursor_next(const DecodeArgs& A, Cursor& c) {
  const int per = c.seg_end - c.base;
  c.base = c.seg_end;
  if (++c.head == A.p.Hkv) {
    c.head = 0;
    ++c.req;
    if (c.req < A.n) cursor_load<UT>(A, c);
  } else {
    c.seg_end = c.base + per;
  }
}

// Columns of the products.  Up to 4 rows: column 2 r is row r's first part and
// 2 r + 1 its second, in one tile (the first product holds the row in both); a
// third part takes the even columns of a second tile.  More rows: column n of
// tile j is row 8 j + n, and the second product has a tile for each part; the small
// parts share one accumulator.
template <int GK, int NR>
struct Cols {
  static constexpr bool DUP = NR <= 4;
  static constexpr int PARTS = GK == 0 ? 3 : 2;
  static constexpr int QT = DUP ? 1 : NR / 8;        // tiles of the first product
  static constexpr int PT = DUP ? PARTS - 1 : PARTS * QT;   // tiles of the second
  static constexpr int OT = DUP ? PT : 2 * QT;       // its accumulators
  __device__ static constexpr int acc(int j) { return DUP ? j : 2 * (j / PARTS) + (j % PARTS ? 1 : 0); }   // of tile j
  static constexpr int HPL = DUP ? 1 : 2;            // rows of a tile that a lane holds
  static constexpr int H = QT * HPL;                 // rows that a lane holds
  // row of the lane's h-th
  __device__ static int row(int h, int tid) { return DUP ? tid : 8 * (h / 2) + 2 * tid + (h & 1); }
};

template <int GK, int NR>
struct State {
  using C = Cols<GK, NR>;
  static constexpr int NG = GK == 64 ? 2 : 1;
  float o[C::OT][8][4];
  float m[C::H], l[C::H];
  float z[NG][C::H];      // sum p z (4 bits)
  int e[NG];              // p s is scaled by 2^(6 - e)
  __device__ void reset() {
#pragma unroll
    for (int i = 0; i < C::OT; ++i)
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][t][k] = 0.0f;
#pragma unroll
    for (int h = 0; h < C::H; ++h) {
      m[h] = NEG_INF;
      l[h] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) z[g][h] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) e[g] = -24;
  }
  // scale row h's accumulators
  __device__ void rescale(int h, float f) {
    l[h] *= f;
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g][h] *= f;
    if constexpr (C::DUP) {
#pragma unroll
      for (int i = 0; i < C::OT; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[i][t][k] *= f;
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          o[2 * (h / 2) + i][t][h & 1] *= f;
          o[2 * (h / 2) + i][t][2 + (h & 1)] *= f;
        }
    }
  }
  // new maximum of row h over the whole warp's tokens
  __device__ void raise(int h, float pm) {
    pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 4));
    pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 8));
    pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 16));
    if (pm > m[h] + LAZY_MAX || (m[h] == NEG_INF && pm > NEG_INF)) {
      rescale(h, m[h] == NEG_INF ? 0.0f : ex2f(m[h] - pm));
      m[h] = pm;
    }
  }
};

// What the row at position pos sees of the 64 tokens from t0; and what any of m rows from
// position pos on sees of them (their windows overlap, or there are only sinks).
__device__ __forceinline__ uint64_t row_sees(const AttnArgs& a, int pos, int t0) {
  return visible_bits(pos - t0, pos - a.window + 1 - t0, a.sinks - t0);
}
__device__ __forceinline__ uint64_t any_sees(const AttnArgs& a, int pos, int m, int t0) {
  return visible_bits(pos + m - 1 - t0, a.window > 0 ? pos - a.window + 1 - t0 : 64, a.sinks - t0);
}

// q as the first product's B operand: column n (= lane / 4), registers of k-step s.
template <int GK, int NR>
struct Query {
  using C = Cols<GK, NR>;
  uint32_t b[C::QT][8][2];
  float scale[C::H];        // softmax scale (x q's power of two in 4 bits) of the lane's rows
  float qsum[GK == 64 ? 2 : 1][C::H];   // 4 bits: sum of q over the group, in the operand's scale
  int pos[C::H];
};

// The segment's query rows into shared memory as the B operand, 16 lanes a row, 8
// channels a lane, by the first NR / 2 warps; take_query() is behind a barrier.  (A warp
// of its own for every row made the same operand twelve times, 7000 cycles of it.)
template <int NR>
__device__ __forceinline__ uint4 load_query(const DecodeArgs& A, int req, int head) {
  const int r = 2 * (threadIdx.x >> 5) + (threadIdx.x >> 4 & 1);
  if (r >= A.m * A.G) return make_uint4(0, 0, 0, 0);
  return *(reinterpret_cast<const uint4*>(A.a.q + (int64_t)(A.req[req].row + r / A.G) * A.a.q_stride +
                                              (int64_t)(head * A.G + r % A.G) * D) + (threadIdx.x & 15));
}
template <int GK, int NR>
__device__ __forceinline__ void put_query(const DecodeArgs& A, uint4 w, DecodeSmem<GK, NR>& sm) {
  using C = Cols<GK, NR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane & 15;
  if (warp >= NR / 2) return;
  const int r = 2 * warp + (lane >> 4);
  if constexpr (GK == 0) {
    // channels 8 part ..: k-step part / 2, register part % 2, one word for each of the four lanes
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (C::DUP) sm.q[0][2 * r][k][part] = sm.q[0][2 * r + 1][k][part] = ww[k];
      else sm.q[r / 8][r % 8][k][part] = ww[k];
    }
  } else {
    // scaled so that the row's largest |q| lies in [2^13, 2^14): exact in fp16 down to 2^-27 of it
    float f[8] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                  __uint_as_float(w.y & 0xffff0000u), __uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u),
                  __uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u)};
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(f[e]));
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    // exponent of the largest, from its bits; not below -112, so that both powers of two are normal
    const int ex = max(-112, static_cast<int>((__float_as_uint(mx) >> 23) & 255) - 127);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + 13 - ex) << 23);
    // (the sum of the scaled channels: that of the channels themselves can overflow)
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] *= up;
      sum += f[e];
    }
#pragma unroll
    for (int off = 1; off < (GK == 128 ? 16 : 8); off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    // the 8 channels are one code word's: codes 2 sub, 2 sub + 1 and those 4 behind
    const uint4 o = make_uint4(f16x2(f[0], f[4]), f16x2(f[1], f[5]), f16x2(f[2], f[6]), f16x2(f[3], f[7]));
    const int tid = GK == 128 ? part / 4 : (part % 8) / 2, word = GK == 128 ? part % 4 : 2 * (part / 8) + part % 2;
    if constexpr (C::DUP)
      *reinterpret_cast<uint4*>(&sm.q[0][2 * r][tid][4 * word]) =
          *reinterpret_cast<uint4*>(&sm.q[0][2 * r + 1][tid][4 * word]) = o;
    else
      *reinterpret_cast<uint4*>(&sm.q[r / 8][r % 8][tid][4 * word]) = o;
    if (part % 8 == 0) {
      // (not 0: it multiplies the -infinity of masked logits)
      sm.q_scale[r] = fmaxf(__uint_as_float(static_cast<uint32_t>(127 + ex - 13) << 23) * A.a.scale2, 1.2e-38f);
      sm.q_sum[part / 8][r] = sum;   // in the operand's scale
    }
  }
}

template <int GK, int NR>
__device__ __forceinline__ void take_query(const DecodeArgs& A, int req, const DecodeSmem<GK, NR>& sm,
                                           Query<GK, NR>& Q) {
  using C = Cols<GK, NR>;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const int first = A.req[req].len - A.m;
#pragma unroll
  for (int j = 0; j < C::QT; ++j)
#pragma unroll
    for (int s = 0; s < 8; s += 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(&sm.q[j][gid][tid][2 * s]);
      Q.b[j][s][0] = w.x, Q.b[j][s][1] = w.y, Q.b[j][s + 1][0] = w.z, Q.b[j][s + 1][1] = w.w;
    }
#pragma unroll
  for (int h = 0; h < C::H; ++h) {
    const int r = C::row(h, tid);
    Q.pos[h] = first + min(r, A.m * A.G - 1) / A.G;
    Q.scale[h] = GK == 0 ? A.a.scale2 : sm.q_scale[r];
    if constexpr (GK != 0) {
#pragma unroll
      for (int g = 0; g < (GK == 64 ? 2 : 1); ++g) Q.qsum[g][h] = sm.q_sum[g][r];
    }
  }
}

// B operand of the second product from the weights of the lane's rows: w0[h] and
// w1[h] for tokens gid and gid + 8 of a 16-token tile.  P: the parts' type (pack rounds
// two values to it, lo and hi give them back).
template <int GK, int NR, typename P>
__device__ __forceinline__ void weights(const float (&w0)[Cols<GK, NR>::H], const float (&w1)[Cols<GK, NR>::H],
                                        uint32_t (&b)[Cols<GK, NR>::PT][2], P) {
  using C = Cols<GK, NR>;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float (&w)[C::H] = u ? w1 : w0;
    if constexpr (C::DUP) {
      const float h = P::round(w[0]), l = w[0] - h;
      b[0][u] = movmatrix(P::pack(h, l));
      if constexpr (C::PARTS == 3) b[1][u] = movmatrix(P::pack(l - P::round(l), 0.0f));
    } else {
#pragma unroll
      for (int j = 0; j < C::QT; ++j) {
        float a = w[2 * j], c = w[2 * j + 1];
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part) {
          const uint32_t both = P::pack(a, c);
          b[C::PARTS * j + part][u] = movmatrix(both);
          a -= P::lo(both);
          c -= P::hi(both);
        }
      }
    }
  }
}
struct PartsBf16 {
  __device__ static float round(float x) { return bf16_hi(x); }
  __device__ static uint32_t pack(float a, float b) { return bf16x2(a, b); }
  __device__ static float lo(uint32_t w) { return __uint_as_float(w << 16); }
  __device__ static float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
};
struct PartsF16 {
  __device__ static float round(float x) { return f16_hi(x); }
  __device__ static uint32_t pack(float a, float b) { return f16x2(a, b); }
  __device__ static float lo(uint32_t w) { return __low2float(*reinterpret_cast<const __half2*>(&w)); }
  __device__ static float hi(uint32_t w) { return __high2float(*reinterpret_cast<const __half2*>(&w)); }
};

// One unit of 16 BF16 tokens from t0: stage = two halves of 64 channels, each K
// [16][128 B] and V [16][128 B], 16-byte pieces swizzled within 8 rows by the TMA.
template <int NR>
__device__ __forceinline__ void bf16_unit(const DecodeArgs& A, const Query<0, NR>& Q, State<0, NR>& S, uint8_t* stage,
                                          int t0, bool masked) {
  using C = Cols<0, NR>;
  const int lane = threadIdx.x & 31, gid = lane >> 2;
  if (masked) {
    // value rows that no row of the segment sees may hold anything: zero them
    const int row = lane & 15, p0 = __shfl_sync(0xffffffffu, Q.pos[0], 0);   // the first query token
    if (!(any_sees(A.a, p0, A.m, t0) >> row & 1)) {
      uint4* v = reinterpret_cast<uint4*>(stage + (lane >> 4) * 4096 + 2048 + row * 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
  }
  const uint32_t base = smem_u32(stage);
  float s[C::QT][4];
#pragma unroll
  for (int j = 0; j < C::QT; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[j][k] = 0.0f;
  const int krow = lane & 15, kc = lane >> 4;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    uint32_t af[4];
    ldsm4(af, base + (ks >> 2) * 4096 + krow * 128 + (((2 * (ks & 3) + kc) ^ (krow & 7)) << 4));
#pragma unroll
    for (int j = 0; j < C::QT; ++j) mma_bf16(s[j], af, Q.b[j][ks][0], Q.b[j][ks][1]);
  }
  float x0[C::H], x1[C::H];
#pragma unroll
  for (int h = 0; h < C::H; ++h) {
    x0[h] = s[h / C::HPL][h % C::HPL] * Q.scale[h];
    x1[h] = s[h / C::HPL][2 + h % C::HPL] * Q.scale[h];
    if (masked) {
      const uint32_t see = static_cast<uint32_t>(row_sees(A.a, Q.pos[h], t0)) >> gid;
      if (!(see & 1)) x0[h] = NEG_INF;
      if (!(see & 0x100)) x1[h] = NEG_INF;
    }
    S.raise(h, fmaxf(x0[h], x1[h]));
    const float ref = S.m[h] == NEG_INF ? 0.0f : S.m[h];
    x0[h] = ex2f(x0[h] - ref);
    x1[h] = ex2f(x1[h] - ref);
    S.l[h] += x0[h] + x1[h];
  }
  uint32_t b[C::PT][2];
  weights<0, NR>(x0, x1, b, PartsBf16());
  const int vrow = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    uint32_t af[4];
    ldsm4_t(af, base + (mt >> 2) * 4096 + 2048 + vrow * 128 + (((2 * (mt & 3) + vc) ^ (vrow & 7)) << 4));
#pragma unroll
    for (int j = 0; j < C::PT; ++j) mma_bf16(S.o[C::acc(j)][mt], af, b[j][0], b[j][1]);
  }
}

// Codes (bits 0-3 and 16-19, or 4-7 and 20-23, of w) as a pair of fp16 numbers c - 8.
// magic (0x64006400: 1024, twice) comes in a register: as a constant beside the mask it
// would cost a second logic operation.
__device__ __forceinline__ uint32_t code_lo(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(magic));   // 1024 + c
  asm("add.rn.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xE408E408u));                    // - 1032
  return x;
}
__device__ __forceinline__ uint32_t code_hi(uint32_t w, uint32_t magic) {
  uint32_t x;
  asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(magic));   // 1024 + 16 c
  asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(x) : "r"(0x2C002C00u), "r"(0xD480D480u));   // / 16 - 72
  return x;
}

// One 4-bit page (64 tokens from t0) as it lies in memory.  Row r of a 16-token tile is
// token r ^ ((r >> 1) & 1), which spreads both products' reads over the banks.
template <int GK, int NR>
__device__ __forceinline__ void int4_unit(const DecodeArgs& A, const Query<GK, NR>& Q, State<GK, NR>& S,
                                          uint8_t* stage, int t0, bool masked) {
  using C = Cols<GK, NR>;
  constexpr int NG = State<GK, NR>::NG, TILES = PAGE / 16, MROW = i4_meta_row(GK);
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
  const int tok = gid ^ ((gid >> 1) & 1);
  uint32_t magic = 0x64006400u;
  asm volatile("" : "+r"(magic));
  if (masked) {
    // the scale and zero of a token that no row sees may be anything: zero them (its codes
    // are finite whatever they are)
    const uint64_t any = any_sees(A.a, __shfl_sync(0xffffffffu, Q.pos[0], 0), A.m, t0);
#pragma unroll 1
    for (int slot = lane; slot < PAGE; slot += 32) {
      if (any >> slot & 1) continue;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        *reinterpret_cast<uint32_t*>(stage + I4_META + MROW * slot + 4 * g) = 0;
        *reinterpret_cast<uint32_t*>(stage + i4_v_meta(GK) + MROW * slot + 4 * g) = 0;
      }
    }
    fence_async_smem();
    __syncwarp();
  }
  // ---- logits of the page
  float x[TILES][2][C::H];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    float s[C::QT][2][4];
#pragma unroll
    for (int j = 0; j < C::QT; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][0][k] = s[j][1][k] = 0.0f;
    uint32_t w[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* row = stage + (16 * t + 8 * u + tok) * I4_ROW;
      if constexpr (GK == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * tid);
        w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
      } else {
        // (two-way bank conflicts; putting them right took two selects a word)
        const uint2 va = *reinterpret_cast<const uint2*>(row + 8 * tid);
        const uint2 vb = *reinterpret_cast<const uint2*>(row + 32 + 8 * tid);
        w[u][0] = va.x, w[u][1] = va.y, w[u][2] = vb.x, w[u][3] = vb.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int g = 0; g < 2; ++g) {   // the two accumulators (groups, at 64) in turn
          const int word = 2 * g + i;
          const uint32_t wa = w[0][word] >> (8 * sub), wb = w[1][word] >> (8 * sub);
          const uint32_t a0 = code_lo(wa, magic), a1 = code_lo(wb, magic), a2 = code_hi(wa, magic), a3 = code_hi(wb, magic);
#pragma unroll
          for (int j = 0; j < C::QT; ++j)
            mma_f16(s[j][g], a0, a1, a2, a3, Q.b[j][2 * word + sub][0], Q.b[j][2 * word + sub][1]);
        }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int slot = 16 * t + 8 * u + tok;
      float sk[2], zk[2];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const __half2 m = *reinterpret_cast<const __half2*>(stage + I4_META + MROW * slot + 4 * g);
        sk[g] = __low2float(m);
        zk[g] = fmaf(8.0f, sk[g], __high2float(m));
      }
#pragma unroll
      for (int h = 0; h < C::H; ++h) {
        const int j = h / C::HPL, k = 2 * u + h % C::HPL;
        float y;
        if constexpr (NG == 1)
          y = fmaf(sk[0], s[j][0][k] + s[j][1][k], zk[0] * Q.qsum[0][h]);
        else
          y = fmaf(sk[0], s[j][0][k], fmaf(sk[1], s[j][1][k], fmaf(zk[0], Q.qsum[0][h], zk[1] * Q.qsum[1][h])));
        x[t][u][h] = y;
      }
    }
  }
  if (masked) {
#pragma unroll
    for (int h = 0; h < C::H; ++h) {
      const uint64_t see = row_sees(A.a, Q.pos[h], t0) >> tok;
      const uint32_t part[2] = {static_cast<uint32_t>(see), static_cast<uint32_t>(see >> 32)};
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (!(part[t / 2] >> (16 * (t % 2) + 8 * u) & 1)) x[t][u][h] = NEG_INF;
    }
  }
#pragma unroll
  for (int h = 0; h < C::H; ++h) {
    float pm = NEG_INF;
#pragma unroll
    for (int t = 0; t < TILES; ++t) pm = fmaxf(pm, fmaxf(x[t][0][h], x[t][1][h]));
    S.raise(h, pm * Q.scale[h]);
    const float ref = S.m[h] == NEG_INF ? 0.0f : -S.m[h];
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x[t][u][h] = ex2f(fmaf(x[t][u][h], Q.scale[h], ref));
        S.l[h] += x[t][u][h];
      }
  }
  // ---- the value scales' power of two: their largest in the page
  const uint8_t* vmeta = stage + i4_v_meta(GK);
  float mult[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t b0 = *reinterpret_cast<const uint16_t*>(vmeta + MROW * lane + 4 * g),
                   b1 = *reinterpret_cast<const uint16_t*>(vmeta + MROW * (lane + 32) + 4 * g);
    uint32_t big = max(b0 & 0x7fffu, b1 & 0x7fffu);
    big = __reduce_max_sync(0xffffffffu, big);
    // s < 2^e: normal numbers have e = (bits >> 10) - 14, subnormal ones e <= -14
    const int e = max(S.e[g], big >= 0x400u ? static_cast<int>(big >> 10) - 14 : (big ? -14 : -24));
    if (e > S.e[g]) {
      const float f = __uint_as_float(static_cast<uint32_t>(127 + S.e[g] - e) << 23);
#pragma unroll
      for (int j = 0; j < C::PT; ++j)
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
          if (NG == 1 || mt / 4 == g)
#pragma unroll
            for (int k = 0; k < 4; ++k) S.o[j][mt][k] *= f;
      S.e[g] = e;
    }
    mult[g] = __uint_as_float(static_cast<uint32_t>(127 + 6 - e) << 23);
  }
  // ---- values
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    uint32_t b[NG][C::PT][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float w0[C::H], w1[C::H];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int slot = 16 * t + 8 * u + tok;
        const __half2 m = *reinterpret_cast<const __half2*>(vmeta + MROW * slot + 4 * g);
        const float sv = __low2float(m) * mult[g], zv = fmaf(8.0f, __low2float(m), __high2float(m));
#pragma unroll
        for (int h = 0; h < C::H; ++h) {
          const float pr = x[t][u][h];
          (u ? w1[h] : w0[h]) = pr * sv;
          S.z[g][h] = fmaf(pr, zv, S.z[g][h]);
        }
      }
      weights<GK, NR>(w0, w1, b[g], PartsF16());
    }
    // the lane's four tokens of the tile: rows 2 tid, 2 tid + 1, + 8; two words of 8
    // channels of each (at group 64 one of each group)
    uint32_t v[4][2];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 2 * tid + (q & 1) + 8 * (q >> 1);
      const uint8_t* row = stage + I4_V_CODES + (16 * t + (r ^ ((r >> 1) & 1))) * I4_ROW;
      if constexpr (GK == 128) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 8 * gid);
        v[q][0] = w.x, v[q][1] = w.y;
      } else {
        v[q][0] = *reinterpret_cast<const uint32_t*>(row + 4 * gid);
        v[q][1] = *reinterpret_cast<const uint32_t*>(row + 32 + 4 * gid);
      }
    }
#pragma unroll
    for (int word = 0; word < 2; ++word)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7632u : 0x5410u;
        const uint32_t pa = __byte_perm(v[0][word], v[1][word], sel), pb = __byte_perm(v[2][word], v[3][word], sel);
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const uint32_t qa = pa >> (8 * sub), qb = pb >> (8 * sub);
          const uint32_t a0 = code_lo(qa, magic), a1 = code_hi(qa, magic), a2 = code_lo(qb, magic), a3 = code_hi(qb, magic);
          const int mt = 4 * word + 2 * half + sub;
#pragma unroll
          for (int j = 0; j < C::PT; ++j)
            mma_f16(S.o[j][mt], a0, a1, a2, a3, b[NG == 1 ? 0 : word][j][0], b[NG == 1 ? 0 : word][j][1]);
        }
      }
  }
}

// This warp's state into shared memory: o in channel order, m, l.
template <int GK, int NR>
__device__ __forceinline__ void put_state(const State<GK, NR>& S, float (*st)[PARTIAL_FLOATS]) {
  using C = Cols<GK, NR>;
  constexpr int NG = State<GK, NR>::NG;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
#pragma unroll
  for (int h = 0; h < C::H; ++h) {
    float l = S.l[h], z[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) z[g] = S.z[g][h];
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
      for (int g = 0; g < NG; ++g) z[g] += __shfl_xor_sync(0xffffffffu, z[g], off);
    }
    const int r = C::row(h, tid);
    if (r >= NR) continue;
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      float a, b;
      if constexpr (C::DUP) {
        a = S.o[0][mt][0] + S.o[0][mt][1];
        b = S.o[0][mt][2] + S.o[0][mt][3];
        if constexpr (C::PARTS == 3) {
          a += S.o[1][mt][0];
          b += S.o[1][mt][2];
        }
      } else {
        const int j = 2 * (h / 2), k = h & 1;
        a = S.o[j][mt][k] + S.o[j + 1][mt][k];
        b = S.o[j][mt][2 + k] + S.o[j + 1][mt][2 + k];
      }
      if constexpr (GK == 0) {
        st[r][16 * mt + gid] = a;
        st[r][16 * mt + gid + 8] = b;
      } else {
        const int g = NG == 1 ? 0 : mt / 4;
        const float back = __uint_as_float(static_cast<uint32_t>(127 + S.e[g] - 6) << 23);
        const int ch = GK == 128 ? 16 * gid + 2 * mt : 64 * (mt / 4) + 8 * gid + 2 * (mt % 4);
        st[r][ch] = fmaf(a, back, z[g]);
        st[r][ch + 1] = fmaf(b, back, z[g]);
      }
    }
    if (gid == 0) {
      st[r][PARTIAL_M] = S.m[h];
      st[r][PARTIAL_L] = l;
    }
  }
}

__device__ __forceinline__ void write_row(const DecodeArgs& A, int req, int head, int r, int lane, float4 o, float m,
                                          float l) {
  const size_t row = (size_t)(A.req[req].row + r / A.G) * A.a.Hq + (size_t)head * A.G + r % A.G;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
  if (A.a.f32) {
    reinterpret_cast<float4*>(static_cast<float*>(A.a.out) + row * D)[lane] = o;
  } else {
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.a.out) + row * D)[lane] =
        make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
  }
  if (A.a.lse && lane == 0) A.a.lse[row] = l != 0.0f ? (m + log2f(l)) * 0.6931471805599453f : NEG_INF;
}

// Fold count states of one row, the warp's lanes holding 4 channels each: weights by 32
// lanes at once, rows FOLD_ROWS at a time, the first of them on their way with the weights.
// The code runs once in a launch, from a cold instruction cache, so it is short.
constexpr int FOLD_ROWS = 8;   // (16: the same times)
template <typename P>
__device__ __forceinline__ void fold(int count, P at, int lane, float4& o, float& m, float& l) {
  m = NEG_INF;
  l = 0.0f;
  o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int base = 0; base < count; base += 32) {
    const float* mine = at(min(base + lane, count - 1));
    const float mc = base + lane < count ? __ldcg(mine + PARTIAL_M) : NEG_INF, lc = __ldcg(mine + PARTIAL_L);
    float f = 0.0f;
#pragma unroll 1
    for (int c = 0; c < 32 && base + c < count; c += FOLD_ROWS) {
      float4 v[FOLD_ROWS];
#pragma unroll
      for (int u = 0; u < FOLD_ROWS; ++u)
        v[u] = __ldcg(reinterpret_cast<const float4*>(at(min(base + c + u, count - 1))) + lane);
      if (c == 0) {
        float top = fmaxf(mc, m);
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float ref = top == NEG_INF ? 0.0f : top, f0 = ex2f(m - ref);
        f = ex2f(mc - ref);
        float sum = lc * f;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = fmaf(l, f0, sum);
        m = top;
        o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
      }
#pragma unroll
      for (int u = 0; u < FOLD_ROWS; ++u) {
        const float w = __shfl_sync(0xffffffffu, f, c + u);   // 0 behind the last
        o.x = fmaf(v[u].x, w, o.x);
        o.y = fmaf(v[u].y, w, o.y);
        o.z = fmaf(v[u].z, w, o.z);
        o.w = fmaf(v[u].w, w, o.w);
      }
    }
  }
}

template <int GK, int NR>
__global__ void __launch_bounds__(DecodeShape<GK, NR>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ DecodeArgs A, const __grid_constant__ CUtensorMap map) {
  using F = Format<GK>;
  using SM = DecodeSmem<GK, NR>;
  constexpr int UT = F::UT, STAGES = SM::STAGES, NW = SM::NW;
  extern __shared__ uint8_t dec_raw[];
  // (aligned by an offset, not by a cast of the address: the accesses stay shared ones)
  SM& sm = *reinterpret_cast<SM*>(dec_raw + (-smem_u32(dec_raw) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int u0 = static_cast<int>((int64_t)A.total * cta / A.ncta);
  const int u1 = static_cast<int>((int64_t)A.total * (cta + 1) / A.ncta);
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(&sm.full[warp][s], 1);
    mbar_init_fence();
  }
  __syncwarp();
  if (GK == 0 && threadIdx.x == 0) prefetch_map(&map);
  Cursor cc;
  cursor_first<UT>(A, cc, u0);
  grid_dep_launch();
  grid_dep_wait();
  const uint4 q_first = load_query<NR>(A, cc.req, cc.head);   // on its way while the copies are issued

  // ---- the warp's copies: units u0 + warp, + NW, ... of the CTA's range.  Lane l looks
  // up the place of unit 32 k + l of them, so that the page ids of 32 copies come at the
  // price of one; place: record index (-1: nothing to copy) and first token in the page.
  const int mine = u1 - u0 > warp ? (u1 - u0 - warp + NW - 1) / NW : 0;
  int issued = 0, place_rec = -1, place_row = 0;
  bool dead = false;   // a wait gave up: no further copies
  auto issue = [&]() {
    if (issued >= mine || dead) return;
    if ((issued & 31) == 0) {
      place_rec = -1;
      if (issued + lane < mine) {
        Cursor c;
        const int u = u0 + warp + NW * (issued + lane);
        cursor_first<UT>(A, c, u);
        const int v = u - c.base;
        if (v < c.un.units) {
          const int t0 = c.un.unit(v) * UT;
          int32_t page = A.p.table[(size_t)A.req[c.req].table * A.p.max_pages + t0 / PAGE];
          if (page < 0 || page >= A.p.num_pages) {
            if (A.p.err) atomicOr(A.p.err, PAGED_ERR_PAGE);
            page = 0;
          }
          place_rec = page * A.p.Hkv + c.head;
          place_row = t0 % PAGE;
        }
      }
      __syncwarp();
    }
    const int rec = __shfl_sync(0xffffffffu, place_rec, issued & 31);
    const int row = __shfl_sync(0xffffffffu, place_row, issued & 31);
    const int st = issued % STAGES;
    if (lane == 0) {
      uint64_t* full = &sm.full[warp][st];
      if (rec >= 0) {
        uint8_t* dst = sm.ring[warp][st];
        mbar_expect_tx(full, F::BYTES);
        if constexpr (GK == 0) {
          tma_load_3d(dst, &map, 0, row, 2 * rec, full);
          tma_load_3d(dst + F::BYTES / 2, &map, 64, row, 2 * rec, full);
        } else {
          tma_load_1d(dst, static_cast<const uint8_t*>(A.p.pool) + (size_t)rec * F::BYTES, F::BYTES, full);
        }
      } else {
        mbar_arrive(full);
      }
    }
    ++issued;
  };
#pragma unroll 1
  for (int s = 0; s < STAGES; ++s) issue();
  put_query<GK, NR>(A, q_first, sm);

  int cu = u0 + warp, taken = 0;
  State<GK, NR> S;
  Query<GK, NR> Q;
  const int R = A.m * A.G;
  for (int seg_u = u0; seg_u < u1;) {
    const int seg_end = min(cc.seg_end, u1);
    if (seg_u > u0) put_query<GK, NR>(A, load_query<NR>(A, cc.req, cc.head), sm);
    __syncthreads();
    take_query<GK, NR>(A, cc.req, sm, Q);
    const int len = A.req[cc.req].len;
    constexpr int MINE = (NR + NW - 1) / NW;   // rows of a warp
    float4 fo[MINE];
    float fm[MINE], fl[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      fo[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      fm[i] = NEG_INF;
      fl[i] = 0.0f;
    }
    // A share of more than 256 units a warp is taken in parts, since the matrix unit
    // truncates its sums: 20 requests of 60K, error 6.2e-6 at once and 4.0e-6 in parts, plain
    // fp32 4.5e-6, the same 702 us.  (Not where the sums in between cost more registers than
    // there are: 16 rows 752 against 718 us; 4 bits 245 against 238 us, error 4.7e-6 against
    // 5.1e-6.)
    constexpr bool PARTS = GK == 0 && NR <= 8;
    constexpr int PART = 256 * NW;
    int part_u = seg_u;
    do {
      const int part_end = PARTS && seg_end - part_u > PART ? part_u + PART : seg_end;
      S.reset();
      for (; cu < part_end; cu += NW) {
        const int v = cu - cc.base, st = taken % STAGES;
        if (!dead && !mbar_wait(&sm.full[warp][st], (taken / STAGES) & 1)) {
          if (lane == 0 && A.p.err) atomicOr(A.p.err, PAGED_ERR_TIMEOUT);
          dead = true;
        }
        dead = __any_sync(0xffffffffu, dead);
        if (!dead && v < cc.un.units) {
          const int t0 = cc.un.unit(v) * UT;
          const bool masked = !(t0 + UT - 1 <= len - A.m &&
                                (t0 + UT <= A.a.sinks || (int64_t)t0 > (int64_t)len - 1 - A.a.window));
          if constexpr (GK == 0)
            bf16_unit<NR>(A, Q, S, sm.ring[warp][st], t0, masked);
          else
            int4_unit<GK, NR>(A, Q, S, sm.ring[warp][st], t0, masked);
        }
        __syncwarp();
        ++taken;
        issue();
      }
      // ---- the CTA's share of the segment: the warps' states folded a few at a time
      // (all of them at once would take the ring's room)
      constexpr int FOLD = SM::FOLD;
      using StateRows = float (*)[PARTIAL_FLOATS];
      static_assert(sizeof(float) * NR * PARTIAL_FLOATS <= sizeof(sm.ring[0]), "a state fits its warp's ring");
      const bool final_seg = part_end == u1;   // no copy is in flight: every warp's state over its own ring, at once
      const int step = final_seg ? NW : FOLD;
#pragma unroll 1
      for (int w0 = 0; w0 < NW; w0 += step) {
        if (warp >= w0 && warp < w0 + step)
          put_state<GK, NR>(S, final_seg ? reinterpret_cast<StateRows>(sm.ring[warp][0]) : sm.state[warp - w0]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          const int r = warp + NW * i;
          if (r >= R) continue;
          float4& o = fo[i];
#pragma unroll 2
          for (int w = 0; w < step; ++w) {
            const float* st = final_seg ? reinterpret_cast<StateRows>(sm.ring[w][0])[r] : sm.state[w][r];
            const float ms = st[PARTIAL_M], m = fmaxf(fm[i], ms), ref = m == NEG_INF ? 0.0f : m;
            const float f0 = ex2f(fm[i] - ref), f = ex2f(ms - ref);
            const float4 x = reinterpret_cast<const float4*>(st)[lane];
            fm[i] = m;
            fl[i] = fmaf(st[PARTIAL_L], f, fl[i] * f0);
            o.x = fmaf(x.x, f, o.x * f0);
            o.y = fmaf(x.y, f, o.y * f0);
            o.z = fmaf(x.z, f, o.z * f0);
            o.w = fmaf(x.w, f, o.w * f0);
          }
        }
        if (!final_seg) __syncthreads();
      }
      part_u = part_end;
    } while (PARTS && part_u < seg_end);
    const int full_units = cc.seg_end - cc.base;
    const int seg = cc.req * A.p.Hkv + cc.head;
    const int c_lo = static_cast<int>((((int64_t)cc.base + 1) * A.ncta - 1) / A.total);
    const int c_hi = static_cast<int>(((int64_t)cc.seg_end * A.ncta - 1) / A.total);
    const bool whole = seg_end - seg_u == full_units;
    float* rec = A.partials + (size_t)(seg + cta) * NR * PARTIAL_FLOATS;
#pragma unroll
    for (int i = 0; i < MINE; ++i) {
      const int r = warp + NW * i;
      if (r >= R) continue;
      if (whole) {
        write_row(A, cc.req, cc.head, r, lane, fo[i], fm[i], fl[i]);
      } else {
        reinterpret_cast<float4*>(rec + r * PARTIAL_FLOATS)[lane] = fo[i];
        if (lane == 0) {
          rec[r * PARTIAL_FLOATS + PARTIAL_M] = fm[i];
          rec[r * PARTIAL_FLOATS + PARTIAL_L] = fl[i];
        }
      }
    }
    if (!whole) {
      // the last CTA of the segment to get here folds its records
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) sm.last = atomicAdd(A.counters + seg, 1) == c_hi - c_lo;
      __syncthreads();
      if (sm.last) {
        __threadfence();
        const float* first = A.partials + (size_t)(seg + c_lo) * NR * PARTIAL_FLOATS;
        for (int r = warp; r < R; r += NW) {
          float4 o;
          float m, l;
          fold(c_hi - c_lo + 1,
               [&](int c) { return first + ((size_t)c * NR + r) * PARTIAL_FLOATS; }, lane, o, m, l);
          write_row(A, cc.req, cc.head, r, lane, o, m, l);
        }
        if (threadIdx.x == 0) A.counters[seg] = 0;
      }
    }
    __syncthreads();   // the states and the flag are free
    seg_u = seg_end;
    if (seg_u < u1) cursor_next<UT>(A, cc);
  }
  // a warp that gave up leaves no copy in flight behind (bounded again)
  if (dead)
    for (; taken < issued; ++taken) mbar_wait(&sm.full[warp][taken % STAGES], (taken / STAGES) & 1);
}

template <int GK, int NR>
cudaError_t launch_decode_t(DecodeArgs& A, const CUtensorMap& map, int sms, cudaStream_t s) {
  constexpr int bytes = static_cast<int>(sizeof(DecodeSmem<GK, NR>)) + 1024;
  static std::atomic<unsigned> done{0};   // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 32 || !(done.load() & (1u << dev))) {
    e = cudaFuncSetAttribute(paged_decode_kernel<GK, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev < 32) done.fetch_or(1u << dev);
  }
  // One CTA per SM; where a CTA's warps would have no unit each, fewer; and one per
  // segment where that leaves its warps at most three units, since folding a segment's
  // CTAs takes longer than two units.
  constexpr int NW = DecodeShape<GK, NR>::NW;
  const int most = (A.total - 1) / NW + 1, segments = A.n * A.p.Hkv;
  int ctas = most < sms ? most : sms;
  if (segments <= sms && A.total <= 3 * NW * segments) ctas = segments;
  A.ncta = ctas;
  return launch_dependent(paged_decode_kernel<GK, NR>, ctas, DecodeShape<GK, NR>::THREADS, bytes, s, A, map);
}

template <int GK>
cudaError_t launch_decode_g(DecodeArgs& A, const CUtensorMap& map, int sms, cudaStream_t s) {
  const int R = A.m * A.G;
  if (R <= 4) return launch_decode_t<GK, 4>(A, map, sms, s);
  if (R <= 8) return launch_decode_t<GK, 8>(A, map, sms, s);
  return launch_decode_t<GK, 16>(A, map, sms, s);
}

int row_class(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

}  // namespace

size_t paged_decode_record_bytes(int segments, int rows, int sms) {
  return (size_t)(segments + sms) * row_class(rows) * PARTIAL_FLOATS * sizeof(float);
}

int64_t paged_decode_units(const AttnReq& r, const AttnArgs& a, int gk, int hkv) {
  const Units u = Units::of(r.len, r.m, a.window, a.sinks, gk == 0 ? Format<0>::UT : PAGE);
  return (int64_t)hkv * (u.units > 0 ? u.units : 1);
}

cudaError_t launch_paged_decode(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a, int gk,
                                void* workspace, const CUtensorMap* map, int sms, cudaStream_t s) {
  DecodeArgs A;
  A.p = p;
  A.a = a;
  A.n = n;
  A.m = reqs[0].m;
  A.G = a.Hq / p.Hkv;
  A.counters = static_cast<int32_t*>(workspace);
  A.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + PAGED_COUNTER_BYTES);
  const int ut = gk == 0 ? Format<0>::UT : PAGE;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    const Units u = Units::of(reqs[i].len, A.m, a.window, a.sinks, ut);
    A.req[i] = {reqs[i].len, reqs[i].row, reqs[i].table, static_cast<int32_t>(total), u};
    total += paged_decode_units(reqs[i], a, gk, p.Hkv);
    if (total > DECODE_MAX_UNITS) return cudaErrorInvalidValue;
  }
  A.total = static_cast<int32_t>(total);
  static const CUtensorMap none = {};
  const CUtensorMap& m = map ? *map : none;
  if (gk == 0) return launch_decode_g<0>(A, m, sms, s);
  if (gk == 128) return launch_decode_g<128>(A, m, sms, s);
  return launch_decode_g<64>(A, m, sms, s);
}

}  // namespace oscar
