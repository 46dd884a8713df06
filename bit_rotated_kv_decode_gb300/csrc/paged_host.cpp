// Host entry points of the paged-cache operators: argument checks, the tensor map
// of a BF16 pool, row and launch planning.  Nothing is allocated and nothing
// throws; every check is made before the first launch.
#include <cmath>
#include <cstdio>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "oscar.h"
#include "paged.h"

using namespace oscar;

namespace {

thread_local char g_message[256] = "";

oscar_status fail(oscar_status st, const char* what) {
  std::snprintf(g_message, sizeof g_message, "%s", what);
  return st;
}
oscar_status bad(const char* what) { return fail(OSCAR_ERR_INVALID_ARG, what); }
oscar_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return OSCAR_OK;
  std::snprintf(g_message, sizeof g_message, "launch: %s", cudaGetErrorString(e));
  return OSCAR_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Checks shared by every call; null if they hold.
const char* check_pages(const void* pool, int64_t num_pages, const int32_t* table, int32_t max_pages, int32_t n,
                        int32_t hkv, const int32_t* error) {
  if (!pool || !aligned16(pool)) return "null or misaligned page pool";
  if (!table || !aligned4(table)) return "null or misaligned page table";
  if (!aligned4(error)) return "misaligned error word";
  if (n < 1 || n > PAGED_MAX_REQ) return "between 1 and 256 requests";
  if (num_pages < 1 || num_pages > INT32_MAX || max_pages < 1) return "bad page counts";
  if (hkv < 1 || hkv > 1024) return "bad number of kv heads";
  if (num_pages * hkv > INT32_MAX / 2) return "pages x kv heads: below 2^30";
  return nullptr;
}

// [pos0, pos0 + count) of every request within its table, rows into r; the number of rows or -1.
int64_t fill_rows(const int32_t* pos0, const int32_t* counts, int32_t n, int32_t max_pages, PagedRows& r) {
  int64_t rows = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t c = counts ? counts[i] : 1;
    // (positions are 32-bit ints in the kernels)
    if (pos0[i] < 0 || c < 0 || (int64_t)pos0[i] + c > (int64_t)PAGE * max_pages || (int64_t)pos0[i] + c > PAGED_MAX_TOKENS)
      return -1;
    r.row0[i] = static_cast<int32_t>(rows);
    r.pos0[i] = pos0[i];
    rows += c;
    if (rows > INT32_MAX / 64) return -1;
  }
  for (int32_t i = n; i <= PAGED_MAX_REQ; ++i) r.row0[i] = static_cast<int32_t>(rows);
  return rows;
}

oscar_status append(void* pool, int64_t num_pages, const int32_t* table, int32_t max_pages, const int32_t* lens,
                    const int32_t* new_lens, int32_t n, int32_t hq, int32_t hkv, int32_t gk, const oscar_rope* rope,
                    const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                    int64_t v_stride, uint16_t* q_out, int32_t* error, void* stream) {
  if (const char* why = check_pages(pool, num_pages, table, max_pages, n, hkv, error)) return bad(why);
  if (!lens) return bad("null lens");
  if (!k || !v || !aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out))
    return bad("null or misaligned q / k / v");
  if ((q == nullptr) != (q_out == nullptr)) return bad("q and q_out come together");
  if (q && (hq < 1 || hq > 8192)) return bad("bad number of query heads");
  const int64_t need_kv = (int64_t)hkv * D;
  if (k_stride < need_kv || v_stride < need_kv || k_stride % 8 || v_stride % 8 ||
      (q && (q_stride < (int64_t)hq * D || q_stride % 8)))
    return bad("a token stride is a multiple of 8 elements and holds the token's heads");
  RopeArgs ra{};
  if (rope) {
    if (!rope->table || !aligned16(rope->table)) return bad("null or misaligned rotation table");
    if (rope->dim < 16 || rope->dim > D || rope->dim % 16) return bad("rotated channels: a multiple of 16, 16 to 128");
    ra.table = rope->table;
    ra.dim = rope->dim;
    ra.interleaved = rope->interleaved != 0;
  }
  PagedRows rows;
  const int64_t total = fill_rows(lens, new_lens, n, max_pages, rows);
  if (total < 0) return bad("lens / new_lens negative, beyond the page table or 2^30 positions");
  if (rope)
    for (int32_t i = 0; i < n; ++i)
      if ((int64_t)lens[i] + (new_lens ? new_lens[i] : 1) > rope->length) return bad("position beyond the rotation table");
  if (total == 0) return OSCAR_OK;
  const PagedView p{pool, table, num_pages, max_pages, n, hkv, error};
  const AppendRows in{q, k, v, q_stride, k_stride, v_stride, q_out, hq};
  return from_cuda(launch_paged_append(p, rows, ra, in, gk, static_cast<cudaStream_t>(stream)));
}

// 3-D view of a BF16 pool: 128 channels, 64 tokens, (page, kv head, K or V).  box:
// 64 channels (the 128-byte swizzle's width) x tokens x parts.
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_entry() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

bool map_3d(CUtensorMap* map, const void* base, cuuint64_t d1, cuuint64_t d2, cuuint64_t stride1, cuuint64_t stride2,
            uint32_t box1, uint32_t box2) {
  const EncodeTiled fn = encode_entry();
  if (!fn) return false;
  const cuuint64_t dims[3] = {D, d1, d2};
  const cuuint64_t strides[2] = {stride1, stride2};   // bytes
  const cuuint32_t box[3] = {64, box1, box2};
  const cuuint32_t steps[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool pool_map(CUtensorMap* map, const void* pool, int64_t records, uint32_t tokens, uint32_t parts) {
  return map_3d(map, pool, PAGE, static_cast<cuuint64_t>(2 * records), D * 2, (cuuint64_t)PAGE * D * 2, tokens, parts);
}

// 3-D view of rows of q, k or v: 128 channels, heads, rows.
bool rows_map(CUtensorMap* map, const void* base, int64_t heads, int64_t rows, int64_t stride, int box_heads,
              int box_rows) {
  return map_3d(map, base, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows), D * 2,
                static_cast<cuuint64_t>(stride) * 2, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_rows));
}

// SMs of the current device; 152 where there is none.
int sm_count() {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 152;
  return sms;
}

bool group_ok(int32_t hq, int32_t hkv) {
  if (hq < 1 || hkv < 1 || hkv > 1024 || hq % hkv) return false;
  const int g = hq / hkv;
  return g == 1 || g == 2 || g == 4 || g == 8;
}

oscar_status attention(const void* pool, int64_t num_pages, const int32_t* table, int32_t max_pages,
                       const int32_t* lens, const int32_t* q_lens, int32_t n, int32_t hq, int32_t hkv, int32_t gk,
                       int32_t window, int32_t sinks, float scale, const uint16_t* q, int64_t q_stride, void* out,
                       int32_t out_type, float* lse, int32_t* error, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (const char* why = check_pages(pool, num_pages, table, max_pages, n, hkv, error)) return bad(why);
  if (!group_ok(hq, hkv)) return bad("query heads per kv head: 1, 2, 4 or 8");
  if (!lens || !q || !out || !workspace) return bad("null lens, q, out or workspace");
  if (!aligned16(q) || !aligned16(out) || !aligned4(lse) || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return bad("misaligned q, out, lse or workspace");
  if (q_stride < (int64_t)hq * D || q_stride % 8) return bad("a token stride is a multiple of 8 elements and holds the token's heads");
  if (out_type != OSCAR_F32 && out_type != OSCAR_BF16) return bad("out is fp32 or bf16");
  if (sinks < 0) return bad("sinks must not be negative");
  if (!std::isfinite(scale)) return bad("scale must be finite");
  const int G = hq / hkv, step = DECODE_MAX_ROWS / G;
  int64_t rows = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t m = q_lens ? q_lens[i] : 1;
    if (m < 0 || lens[i] < m || (int64_t)lens[i] > (int64_t)PAGE * max_pages || lens[i] > PAGED_MAX_TOKENS)
      return bad("0 <= q_lens <= lens <= 64 max_pages, and lens at most 2^30");
    if (gk != 0 && m > step) return bad("4-bit attention: at most 16 / (query heads per kv head) query tokens a request");
    rows += m;
    if (rows > INT32_MAX / 64) return bad("too many query rows");
  }
  if ((int64_t)n * hkv > (int64_t)PAGED_COUNTERS) return bad("requests x kv heads: at most 16384");
  if (workspace_bytes < oscar_attention_workspace_bytes(n, q_lens, hq, hkv)) return bad("workspace too small");
  const PagedView p{const_cast<void*>(pool), table, num_pages, max_pages, n, hkv, error};
  AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.f32 = out_type == OSCAR_F32;
  a.Hq = hq;
  a.window = window < 0 || window > PAGED_MAX_TOKENS ? PAGED_MAX_TOKENS : window;
  a.sinks = sinks;
  a.scale2 = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
  if (!std::isfinite(a.scale2)) return bad("scale too large");
  const int sms = sm_count();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  AttnReq reqs[PAGED_MAX_REQ];
  // requests of more than 16 rows a kv head: the tiled kernel
  int count = 0, few = 0;
  int64_t units = 0;
  int32_t row = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int32_t m = q_lens ? q_lens[i] : 1;
    if (m > step) reqs[count++] = AttnReq{lens[i], m, row, i};
    if (m >= 1 && m <= step) {
      ++few;
      units += paged_decode_units(AttnReq{lens[i], m, row, i}, a, gk, hkv);
    }
    row += m;
  }
  if (units > DECODE_MAX_UNITS) return bad("too many visible tokens for one call");
  CUtensorMap kv_map, q_map;
  if (count) {
    if (!pool_map(&kv_map, pool, num_pages * hkv, PAGE, 1) ||
        !rows_map(&q_map, q, hq, rows, q_stride, G, 128 / G))
      return fail(OSCAR_ERR_CUDA, "tensor map of the pool or of q");
    const cudaError_t e = launch_paged_prefill(p, reqs, count, a, q_map, kv_map,
                                               static_cast<char*>(workspace) + PAGED_COUNTER_BYTES, sms, s);
    if (e != cudaSuccess) return from_cuda(e);
  }
  if (!few) return OSCAR_OK;
  // the others: those of the same number of query tokens go together
  if (gk == 0 && !pool_map(&kv_map, pool, num_pages * hkv, 16, 2))
    return fail(OSCAR_ERR_CUDA, "tensor map of the pool");
  for (int32_t m = step; m >= 1 && few; --m) {
    count = 0;
    row = 0;
    for (int32_t i = 0; i < n; ++i) {
      const int32_t mi = q_lens ? q_lens[i] : 1;
      if (mi == m) reqs[count++] = AttnReq{lens[i], m, row, i};
      row += mi;
    }
    if (!count) continue;
    few -= count;
    const cudaError_t e = launch_paged_decode(p, reqs, count, a, gk, workspace, gk == 0 ? &kv_map : nullptr, sms, s);
    if (e != cudaSuccess) return from_cuda(e);
  }
  return OSCAR_OK;
}

// Lengths of packed sequences: their rows in all, or -1; their row blocks for an output type.
int64_t packed_rows(const int32_t* lens, int32_t n) {
  int64_t rows = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (lens[i] < 0 || lens[i] > PAGED_MAX_TOKENS) return -1;
    rows += lens[i];
    if (rows > INT32_MAX / 64) return -1;
  }
  return rows;
}
size_t prompt_bytes(const int32_t* lens, int32_t n, int G, int hkv, bool f32, int sms) {
  int64_t blocks = 0;
  for (int32_t i = 0; i < n; ++i) blocks += paged_prefill_blocks(lens[i], G, f32);
  return 256 + paged_prefill_partial_bytes(blocks, hkv, sms, f32);
}

oscar_status prompt(const int32_t* lens, int32_t n, int32_t hq, int32_t hkv, int32_t window, int32_t sinks, float scale,
                    const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                    int64_t v_stride, void* out, int32_t out_type, float* lse, int32_t* error, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (n < 1 || n > PAGED_MAX_REQ) return bad("between 1 and 256 sequences");
  if (!group_ok(hq, hkv)) return bad("query heads per kv head: 1, 2, 4 or 8");
  if (!lens) return bad("null lens");
  if (!q || !k || !v || !out || !workspace) return bad("null q, k, v, out or workspace");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(lse) || !aligned4(error) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255))
    return bad("misaligned q, k, v, out, lse, error or workspace");
  const int64_t need_kv = (int64_t)hkv * D, most = (int64_t)1 << 38;   // (a tensor map's strides stay below 2^40 bytes)
  if (q_stride < (int64_t)hq * D || k_stride < need_kv || v_stride < need_kv || q_stride % 8 || k_stride % 8 ||
      v_stride % 8 || q_stride > most || k_stride > most || v_stride > most)
    return bad("a token stride is a multiple of 8 elements and holds the token's heads");
  if (out_type != OSCAR_F32 && out_type != OSCAR_BF16) return bad("out is fp32 or bf16");
  if (sinks < 0) return bad("sinks must not be negative");
  if (!std::isfinite(scale)) return bad("scale must be finite");
  const int64_t rows = packed_rows(lens, n);
  if (rows < 0) return bad("lens negative, or too many rows");
  AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.out = out;
  a.lse = lse;
  a.f32 = out_type == OSCAR_F32;
  a.Hq = hq;
  a.window = window < 0 || window > PAGED_MAX_TOKENS ? PAGED_MAX_TOKENS : window;
  a.sinks = sinks;
  a.scale2 = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
  if (!std::isfinite(a.scale2)) return bad("scale too large");
  const int G = hq / hkv, sms = sm_count();
  if (workspace_bytes < prompt_bytes(lens, n, G, hkv, a.f32, sms)) return bad("workspace too small");
  if (rows == 0) return OSCAR_OK;
  AttnReq reqs[PAGED_MAX_REQ];
  int count = 0;
  int32_t row = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (lens[i]) reqs[count++] = AttnReq{lens[i], lens[i], row, 0};
    row += lens[i];
  }
  CUtensorMap q_map, k_map, v_map;
  if (!rows_map(&q_map, q, hq, rows, q_stride, G, 128 / G) || !rows_map(&k_map, k, hkv, rows, k_stride, 1, PAGE) ||
      !rows_map(&v_map, v, hkv, rows, v_stride, 1, PAGE))
    return fail(OSCAR_ERR_CUDA, "tensor map of q, k or v");
  return from_cuda(launch_packed_prefill(reqs, count, hkv, a, q_map, k_map, v_map, error, workspace, sms,
                                         static_cast<cudaStream_t>(stream)));
}

}  // namespace

bool oscar::tensor_map_rows(CUtensorMap* map, const void* base, int64_t heads, int64_t rows, int64_t stride,
                            int box_heads, int box_rows) {
  return rows_map(map, base, heads, rows, stride, box_heads, box_rows);
}
bool oscar::tensor_map_pages(CUtensorMap* map, const void* pool, int64_t records) {
  return pool_map(map, pool, records, PAGE, 1);
}

extern "C" {

const char* oscar_paged_last_error(void) { return g_message; }

oscar_status oscar_bf16_append(void* kv, int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                               const int32_t* lens, const int32_t* new_lens, int32_t n, int32_t num_q_heads,
                               int32_t num_kv_heads, const oscar_rope* rope, const uint16_t* q, int64_t q_stride,
                               const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               uint16_t* q_out, int32_t* error, void* stream) {
  return append(kv, num_pages, page_table, max_pages, lens, new_lens, n, num_q_heads, num_kv_heads, 0, rope, q, q_stride,
                k, k_stride, v, v_stride, q_out, error, stream);
}

oscar_status oscar_int4_append(void* kv, int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                               const int32_t* lens, const int32_t* new_lens, int32_t n, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t group_size, const oscar_rope* rope, const uint16_t* q,
                               int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                               int64_t v_stride, uint16_t* q_out, int32_t* error, void* stream) {
  if (group_size != 128 && group_size != 64) return bad("group_size must be 128 or 64");
  return append(kv, num_pages, page_table, max_pages, lens, new_lens, n, num_q_heads, num_kv_heads, group_size, rope, q,
                q_stride, k, k_stride, v, v_stride, q_out, error, stream);
}

oscar_status oscar_int4_read(const void* kv, int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                             const int32_t* starts, const int32_t* counts, int32_t n, int32_t num_kv_heads,
                             int32_t group_size, void* k_out, void* v_out, int32_t out_type, int32_t* error,
                             void* stream) {
  if (group_size != 128 && group_size != 64) return bad("group_size must be 128 or 64");
  if (const char* why = check_pages(kv, num_pages, page_table, max_pages, n, num_kv_heads, error)) return bad(why);
  if (!starts || !counts || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return bad("null starts or counts, null or misaligned output");
  if (out_type != OSCAR_F32 && out_type != OSCAR_BF16) return bad("out is fp32 or bf16");
  PagedRows rows;
  const int64_t total = fill_rows(starts, counts, n, max_pages, rows);
  if (total < 0) return bad("starts / counts negative, beyond the page table or 2^30 positions");
  if (total == 0) return OSCAR_OK;
  const PagedView p{const_cast<void*>(kv), page_table, num_pages, max_pages, n, num_kv_heads, error};
  return from_cuda(launch_int4_read(p, rows, group_size, k_out, v_out, out_type == OSCAR_F32,
                                    static_cast<cudaStream_t>(stream)));
}

size_t oscar_attention_workspace_bytes(int32_t n, const int32_t* q_lens, int32_t num_q_heads, int32_t num_kv_heads) {
  if (n < 1 || n > PAGED_MAX_REQ || !group_ok(num_q_heads, num_kv_heads) ||
      (int64_t)n * num_kv_heads > (int64_t)PAGED_COUNTERS)
    return 0;
  const int G = num_q_heads / num_kv_heads, sms = sm_count();
  int few = 1;            // most rows of a decode segment
  int64_t blocks[2] = {0, 0};   // row blocks of the longer requests, for bf16 and fp32 outputs
  for (int32_t i = 0; i < n; ++i) {
    const int64_t m = q_lens ? q_lens[i] : 1;
    if (m < 0) return 0;
    if (m * G > DECODE_MAX_ROWS)
      for (int f32 = 0; f32 < 2; ++f32) blocks[f32] += paged_prefill_blocks(static_cast<int>(m), G, f32);
    else if (m * G > few)
      few = static_cast<int>(m) * G;
  }
  // both kernels use the same bytes, one after the other
  size_t most = paged_decode_record_bytes(n * num_kv_heads, few, sms);
  for (int f32 = 0; f32 < 2; ++f32) {
    const size_t prefill = paged_prefill_partial_bytes(blocks[f32], num_kv_heads, sms, f32);
    if (prefill > most) most = prefill;
  }
  return PAGED_COUNTER_BYTES + most;
}

oscar_status oscar_window_attention(const void* kv, int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                                    const int32_t* lens, const int32_t* q_lens, int32_t n, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t window, int32_t sinks, float scale,
                                    const uint16_t* q, int64_t q_stride, void* out, int32_t out_type, float* lse,
                                    int32_t* error, void* workspace, size_t workspace_bytes, void* stream) {
  return attention(kv, num_pages, page_table, max_pages, lens, q_lens, n, num_q_heads, num_kv_heads, 0, window, sinks,
                   scale, q, q_stride, out, out_type, lse, error, workspace, workspace_bytes, stream);
}

oscar_status oscar_int4_attention(const void* kv, int64_t num_pages, const int32_t* page_table, int32_t max_pages,
                                  const int32_t* lens, const int32_t* q_lens, int32_t n, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t group_size, int32_t window, int32_t sinks, float scale,
                                  const uint16_t* q, int64_t q_stride, void* out, int32_t out_type, float* lse,
                                  int32_t* error, void* workspace, size_t workspace_bytes, void* stream) {
  if (group_size != 128 && group_size != 64) return bad("group_size must be 128 or 64");
  return attention(kv, num_pages, page_table, max_pages, lens, q_lens, n, num_q_heads, num_kv_heads, group_size, window,
                   sinks, scale, q, q_stride, out, out_type, lse, error, workspace, workspace_bytes, stream);
}

size_t oscar_prompt_workspace_bytes(int32_t n, const int32_t* lens, int32_t num_q_heads, int32_t num_kv_heads) {
  if (n < 1 || n > PAGED_MAX_REQ || !lens || !group_ok(num_q_heads, num_kv_heads) || packed_rows(lens, n) < 0) return 0;
  const int G = num_q_heads / num_kv_heads, sms = sm_count();
  const size_t b16 = prompt_bytes(lens, n, G, num_kv_heads, false, sms), f32 = prompt_bytes(lens, n, G, num_kv_heads, true, sms);
  return b16 > f32 ? b16 : f32;
}

oscar_status oscar_prompt_attention(const int32_t* lens, int32_t n, int32_t num_q_heads, int32_t num_kv_heads,
                                    int32_t window, int32_t sinks, float scale, const uint16_t* q, int64_t q_stride,
                                    const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, void* out,
                                    int32_t out_type, float* lse, int32_t* error, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  return prompt(lens, n, num_q_heads, num_kv_heads, window, sinks, scale, q, q_stride, k, k_stride, v, v_stride, out,
                out_type, lse, error, workspace, workspace_bytes, stream);
}

}  // extern "C"
