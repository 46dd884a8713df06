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
namespace oscar {
namespace {
// Registers a thread: 168 at launch (three warpgroups share 504), then 208 for the
// softmax's two warpgroups, which hold a row of logits each, and 88 for the third.
constexpr int PF_REGS = 168, PF_SOFTMAX_REGS = 208, PF_OTHER_REGS = 88;
}  // namespace
}  // namespace oscar

#include "paged_prefill_device.cuh"

namespace oscar {

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
  const cudaError_t e = plan(A, p, reqs, n, a, partials, sms, PAGES);
  if (e != cudaSuccess) return e;
  const PrefillMaps maps{q_map, kv_map, {}, {}};
  return launch_source<PAGES>(A, maps, sms, s);
}

}  // namespace oscar
