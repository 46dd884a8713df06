// Declarations of the chunk operators on the three-segment cache: tokens written in
// chunks (extend), read back (read), and attended by a chunk of new tokens.
#pragma once

#include "paged.h"

namespace oscar {

constexpr int CHUNK_MAX_REQ = PAGED_MAX_REQ;   // requests per call: their lengths travel in the kernel arguments

// Request i of an extend: its new tokens are rows row0, row0 + 1, ... of k and v, at the
// positions old, old + 1, ..., end - 1; those of [h0, h1) go to history, the ones below old
// from the ring.
struct ExtendArgs {
  const uint16_t *k, *v;
  int64_t k_stride, v_stride;            // elements from one token's rows to the next
  int n, layer;
  int32_t slot[CHUNK_MAX_REQ];
  int32_t row0[CHUNK_MAX_REQ];
  int32_t old[CHUNK_MAX_REQ];
  int32_t h0[CHUNK_MAX_REQ];
  int32_t h1[CHUNK_MAX_REQ];
  int32_t hist[CHUNK_MAX_REQ + 1];       // history rows before request i
  int32_t rows[CHUNK_MAX_REQ + 1];       // new tokens before request i
};
cudaError_t launch_extend_history(const DevCache& c, const ExtendArgs& a, int sms, cudaStream_t s);
cudaError_t launch_extend_bf16(const DevCache& c, const ExtendArgs& a, cudaStream_t s);

// Request i of a read: its tokens [start, start + count) go to output rows out0 - (first -
// start), ...; those of history are hist[i + 1] - hist[i] from `first` on, at output row out0.
struct ReadArgs {
  void *k_out, *v_out;
  int n, layer;
  int32_t slot[CHUNK_MAX_REQ];
  int32_t start[CHUNK_MAX_REQ];
  int32_t first[CHUNK_MAX_REQ];
  int32_t out0[CHUNK_MAX_REQ];
  int32_t hist[CHUNK_MAX_REQ + 1];       // history rows before request i
  int32_t near[CHUNK_MAX_REQ + 1];       // other rows before request i
};
cudaError_t launch_read_history(const DevCache& c, const ReadArgs& a, bool f32, int sms, cudaStream_t s);
cudaError_t launch_read_bf16(const DevCache& c, const ReadArgs& a, bool f32, cudaStream_t s);

// ---- chunk attention ---------------------------------------------------------------
// q's rows times R_K as fp16, channels in the order that the scan unpacks codes in, each row
// times a power of two whose inverse is its scale.
struct RotateArgs {
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;          // fp16 [rows][Hq][128]
  float* scale;           // [rows][Hq]
  int32_t rows, lg, layer;
};
cudaError_t launch_rotate_queries(const DevCache& c, const RotateArgs& a, int sms, cudaStream_t s);

// The scan's line of work: segment k of request i -- kv head k / blocks, block k % blocks of its rows --
// is setup + tiles units from cost[i] + k (setup + tiles) on, and CTA j has those from cut(j) to cut(j + 1).
// A record of the scan is [2][128 rows][PARTIAL_FLOATS], number segment + CTA (the CTAs that meet a segment
// are neighbours).
constexpr int CHUNK_SETUP = 3;          // a segment's queries and rows of results, in key tiles
struct ScanArgs {
  const float* q_scale;
  float* records;
  int64_t total;                          // units in all
  int32_t ctas, n, layer, setup;
  int32_t Hq, Hkv, G, lg;                 // lg = log2 G
  float scale2;                           // softmax scale x log2(e)
  int32_t slot[CHUNK_MAX_REQ];
  int32_t m[CHUNK_MAX_REQ];               // new tokens
  int32_t row[CHUNK_MAX_REQ];             // first row of q and out
  int32_t hist[CHUNK_MAX_REQ];            // tokens of history
  int32_t tiles[CHUNK_MAX_REQ];           // key tiles
  int32_t blocks[CHUNK_MAX_REQ];          // blocks of rows
  int32_t segment[CHUNK_MAX_REQ];         // segments before
  int64_t cost[CHUNK_MAX_REQ];            // units before
};
__host__ __device__ inline int64_t chunk_cut(const ScanArgs& a, int64_t cta) { return cta * a.total / a.ctas; }
// the CTA that has a unit
__host__ __device__ inline int64_t chunk_of(const ScanArgs& a, int64_t unit) {
  return ((unit + 1) * a.ctas - 1) / a.total;
}
cudaError_t launch_chunk_scan(const DevCache& c, const ScanArgs& a, bool pair, const CUtensorMap& q_map, cudaStream_t s);

// The BF16 tokens' partial rows: [near_blocks from the last][near_splits][Hkv][256 rows][PARTIAL_FLOATS].
struct NearPlan {
  int splits, blocks, ctas;
  int32_t start[CHUNK_MAX_REQ];           // blocks of 256 rows before request i
};
struct MergeArgs {
  const float* near;
  uint16_t* out;
  int32_t near_splits, near_blocks;
  int32_t chunks;                         // pieces of a kv head's rows, and those before request i
  int32_t near_start[CHUNK_MAX_REQ];
  int32_t chunk[CHUNK_MAX_REQ];
};
cudaError_t launch_chunk_merge(const DevCache& c, const ScanArgs& a, MergeArgs& b, bool pair, int sms, cudaStream_t s);

// The BF16 tokens of the cache and the new ones (tensor maps as launch_packed_prefill's and
// launch_paged_prefill's): whole results, or partial rows, of least key tiles or more each.
cudaError_t launch_near_attention(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a, bool partial,
                                  const CUtensorMap& q_map, const CUtensorMap& pool_map, const CUtensorMap& k_map,
                                  const CUtensorMap& v_map, void* partials, int least, NearPlan* plan, int sms, cudaStream_t s);

}  // namespace oscar
