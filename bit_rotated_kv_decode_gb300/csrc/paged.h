// Declarations shared by the paged-cache operators (append with position
// rotation, 4-bit read, windowed attention) and their host entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace oscar {

constexpr int PAGED_MAX_REQ = 256;   // requests per call: their lengths travel in the kernel arguments

constexpr int PAGED_MAX_TOKENS = 1 << 30;   // positions of a request
// A token behind every position; the bounds of what a row sees, taken from it, are ints (the
// first row's window begins at 1 - PAGED_MAX_TOKENS).
constexpr int PAGED_NO_TOKEN = PAGED_MAX_TOKENS;
static_assert(1 - (int64_t)PAGED_MAX_TOKENS - PAGED_NO_TOKEN >= INT32_MIN, "a window's begin less a token is an int");

// error bits of the caller's device word
constexpr int PAGED_ERR_PAGE = 1;      // a page id out of range
constexpr int PAGED_ERR_TIMEOUT = 2;   // a bounded device wait gave up

// 4-bit record of one (page, kv head): K codes [64][64 B], V codes [64][64 B]
// (channel 2j in the low nibble of byte j), K meta [64][128 / group]{fp16 s,
// fp16 z}, V meta the same.
constexpr int I4_ROW = D / 2;
constexpr int I4_V_CODES = PAGE * I4_ROW;
constexpr int I4_META = 2 * PAGE * I4_ROW;
__host__ __device__ constexpr int i4_meta_row(int gk) { return 4 * (D / gk); }
__host__ __device__ constexpr int i4_v_meta(int gk) { return I4_META + PAGE * i4_meta_row(gk); }
__host__ __device__ constexpr int i4_record(int gk) { return I4_META + 2 * PAGE * i4_meta_row(gk); }
static_assert(i4_record(128) == 8704 && i4_record(64) == 9216, "4-bit record sizes");

// Where the pages of n requests are.
struct PagedView {
  void* pool;
  const int32_t* table;   // device [n][max_pages]
  int64_t num_pages;
  int32_t max_pages;
  int32_t n;
  int32_t Hkv;
  int32_t* err;           // device word or null
};

// Rows of a ragged batch: request i has the rows [row0[i], row0[i + 1]), which are
// its positions pos0[i], pos0[i] + 1, ...
struct PagedRows {
  int32_t row0[PAGED_MAX_REQ + 1];
  int32_t pos0[PAGED_MAX_REQ];
};

struct RopeArgs {
  const float* table;     // device fp32 [length][dim]: dim / 2 cosines, then sines; null: no rotation
  int32_t dim;
  int32_t interleaved;
};

struct AppendRows {
  const uint16_t *q, *k, *v;            // bf16; q null: none
  int64_t q_stride, k_stride, v_stride; // elements from one token's rows to the next
  uint16_t* q_out;                      // [rows][Hq][128]
  int32_t Hq;
};

// gk: 0 for BF16 pages, else the quantisation group of 4-bit pages.
cudaError_t launch_paged_append(const PagedView& p, const PagedRows& rows, const RopeArgs& rope, const AppendRows& in,
                                int gk, cudaStream_t s);
cudaError_t launch_int4_read(const PagedView& p, const PagedRows& rows, int gk, void* k_out, void* v_out, bool f32,
                             cudaStream_t s);

// ---- attention ------------------------------------------------------------------
// Request i of the call: its last m positions attend; the query at position p sees
// t <= p with t < sinks or t > p - window.
struct AttnArgs {
  const uint16_t* q;
  int64_t q_stride;
  void* out;
  float* lse;             // or null
  int32_t f32;            // out type
  int32_t Hq;
  int32_t window;         // PAGED_MAX_TOKENS: no bound
  int32_t sinks;
  float scale2;           // softmax scale x log2(e)
};
struct AttnReq {
  int32_t len;            // tokens in the cache, the queries among them
  int32_t m;              // query rows
  int32_t row;            // first row of q / out
  int32_t table;          // row of the page table
};

constexpr size_t PAGED_COUNTERS = 16384;                                  // int32 merge counters, zero between calls
constexpr size_t PAGED_COUNTER_BYTES = PAGED_COUNTERS * sizeof(int32_t);  // at the start of every workspace
constexpr int DECODE_MAX_ROWS = 16;   // query rows (tokens x heads of a group) of one decode segment

// Decode: m * G <= DECODE_MAX_ROWS rows per (request, kv head), the same m for all.
size_t paged_decode_record_bytes(int segments, int rows, int sms);
// Units that a launch takes at most: a warp's index into them steps by the CTA's warps (up to
// 12) past the end of its share, and stays an int.
constexpr int32_t DECODE_MAX_UNITS = INT32_MAX - 64;
int64_t paged_decode_units(const AttnReq& r, const AttnArgs& a, int gk, int hkv);
cudaError_t launch_paged_decode(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a, int gk,
                                void* workspace, const CUtensorMap* map, int sms, cudaStream_t s);

// Prefill: any number of query rows per request, BF16 pages.  q_map: q as (128
// channels, Hq, rows), boxes of 64 channels x G heads x 128 / G rows; kv_map: the pool,
// boxes of 64 channels x 64 tokens x 1.
// partials: paged_prefill_partial_bytes() of the call's row blocks (the sum of
// paged_prefill_blocks()), used where few blocks meet many keys.  f32: fp32 outputs,
// whose blocks are smaller.
int64_t paged_prefill_blocks(int m, int G, bool f32);
size_t paged_prefill_partial_bytes(int64_t blocks, int hkv, int sms, bool f32);
cudaError_t launch_paged_prefill(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a,
                                 const CUtensorMap& q_map, const CUtensorMap& kv_map, void* partials, int sms,
                                 cudaStream_t s);

}  // namespace oscar
