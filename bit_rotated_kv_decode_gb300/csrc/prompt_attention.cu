// Attention of whole prompts within packed sequences, straight from the rows of q, k and v
// that a projection wrote: the tiled kernel of paged_prefill.cu with its keys and values
// loaded as rows (boxes of 64 tokens of one kv head) instead of pages.
namespace oscar {
namespace {
// Registers a thread: 168 at launch (three warpgroups share 504), then 208 for the
// softmax's two warpgroups, which hold a row of logits each, and 88 for the third.
constexpr int PF_REGS = 168, PF_SOFTMAX_REGS = 208, PF_OTHER_REGS = 88;
}  // namespace
}  // namespace oscar

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

}  // namespace oscar
