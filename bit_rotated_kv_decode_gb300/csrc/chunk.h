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

}  // namespace oscar
