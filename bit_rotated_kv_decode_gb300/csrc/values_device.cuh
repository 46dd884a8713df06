// The values z + s c of history tokens as fp16, and tiles of them in shared memory.
#pragma once

#include "tcgen05_device.cuh"

namespace oscar {
namespace paged {

// Values of a kv head are held as x 2^-k with 2^k from 2^8 tau to 2^9 tau (|x| <= tau, s <= 2/3 tau): a
// code's two bits, as the half that they are where they stand in a word, count c 2^(2 at - 24), and
// s 2^(24 - 2 at - k) is a half too, at most 2^16 2/3, so that one fma gives z + s c rounded once.
// What falls below fp16's normal values is then off by at most 2^-17 tau.
__device__ __forceinline__ int value_exponent(float tau) { return static_cast<int>(__float_as_uint(tau) >> 23) - 127 + 9; }
__device__ __forceinline__ float pow2(int e) {   // (thresholds below 2^-100 hold nothing that fp16 can)
  return __uint_as_float(static_cast<uint32_t>(127 + min(max(e, -126), 126)) << 23);
}
// s 2^(24 - 2 at - k) for the places at = 0 ... 4 in a word, and z 2^-k, of a token's {fp16 s, fp16 z}.
__device__ __forceinline__ void value_steps(uint32_t meta, int k, __half2 (&s)[5], __half2& z) {
  const __half2 quarter = __float2half2_rn(0.25f);
  s[0] = __float2half2_rn(__half2float(__ushort_as_half(meta & 0xffff)) * pow2(24 - k));
  z = __float2half2_rn(__half2float(__ushort_as_half(meta >> 16)) * pow2(-k));
#pragma unroll
  for (int j = 1; j < 5; ++j) s[j] = __hmul2(s[j - 1], quarter);
}
// The 16 codes of a word as values: half2 i holds channels i and i + 8 (so position 16 k + 2 i + b of a row
// that is unpacked word by word holds channel 16 k + 8 b + i).
__device__ __forceinline__ void unpack_values(uint32_t w, const __half2 (&s)[5], __half2 z, uint32_t (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = i % 5, shift = 2 * (i - at);
    const uint32_t bits = (w >> shift) & (0x00030003u << (2 * at));
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&bits), s[at], z);
    x[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace paged
}  // namespace oscar
