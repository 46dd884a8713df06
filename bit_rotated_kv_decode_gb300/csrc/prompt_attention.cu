// Attention of whole prompts within packed sequences, straight from the rows of q, k and v
// that a projection wrote: the tiled kernel of paged_prefill.cu with its keys and values
// loaded as rows (boxes of 64 tokens of one kv head) instead of pages.  And the near part of a
// chunk's attention: the same over the three-segment cache's BF16 pages with the chunk's own
// rows behind them.  16K tokens of 32 heads (8 kv heads): 1138 us in runs of 20 calls, 1.93 PFLOP/s; in a loop of
// seconds 1282 to 1312, at the power cap.
namespace oscar {
namespace {
// Registers a thread: 168 at launch (three warpgroups share 504), then 208 for the
// softmax's two warpgroups, which hold a row of logits each, and 88 for the third.
constexpr int PF_REGS = 168, PF_SOFTMAX_REGS = 208, PF_OTHER_REGS = 88;
}  // namespace
}  // namespace oscar

#include "chunk.h"
#include "paged_prefill_device.cuh"

namespace oscar {

cudaError_t launch_packed_prefill(const AttnReq* reqs, int n, int hkv, const AttnArgs& a, const CUtensorMap& q_map,
                                  const CUtensorMap& k_map, const CUtensorMap& v_map, int32_t* err, void* partials,
                                  int sms, cudaStream_t s) {
  PrefillArgs A;
  const PagedView p{nullptr, nullptr, 0, 0, n, hkv, err};
  const cudaError_t e = plan(A, p, reqs, n, a, partials, sms, PACKED);
  if (e != cudaSuccess) return e;
  const PrefillMaps maps{q_map, {}, k_map, v_map};
  return launch_source<PACKED>(A, maps, sms, s);
}

cudaError_t launch_near_attention(const PagedView& p, const AttnReq* reqs, int n, const AttnArgs& a, bool partial,
                                  const CUtensorMap& q_map, const CUtensorMap& pool_map, const CUtensorMap& k_map,
                                  const CUtensorMap& v_map, void* partials, int least, NearPlan* out, int sms, cudaStream_t s) {
  PrefillArgs A;
  const cudaError_t e = plan(A, p, reqs, n, a, partials, sms, CACHE, least);
  if (e != cudaSuccess) return e;
  const PrefillMaps maps{q_map, pool_map, k_map, v_map};
  if (!partial && A.splits == 1) return launch_tiles<false, false, CACHE>(A, maps, sms, s);
  if (!partial) {
    const cudaError_t f = launch_tiles<false, true, CACHE>(A, maps, sms, s);
    return f != cudaSuccess ? f : launch_fold(A, s);
  }
  out->splits = A.splits;
  out->blocks = A.bstart[n];
  out->ctas = A.items < sms ? A.items : sms;
  for (int i = 0; i < n; ++i) out->start[i] = A.bstart[i];
  return launch_tiles<false, true, CACHE>(A, maps, sms, s);
}

}  // namespace oscar
