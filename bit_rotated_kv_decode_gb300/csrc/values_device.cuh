// The values z + s c of history tokens as fp16, and tiles of them in shared memory.
#pragma once

#include "tcgen05_device.cuh"

namespace oscar {
namespace paged {

// Values are held as x 2^-k, with 2^k from 2^8 to 2^9 times the largest of the tokens that share k (3 s is at
// most twice that): a code's two bits, as the half that they are where they stand in a word, count
// c 2^(2 at - 24), and s 2^(24 - 2 at - k) is a half too, at most 2^16 2/3, so that one fma gives z + s c: off
// by 2^-11 of it, its rounding, and by 2^-15 of the largest where it and z fall below fp16's normal values (2^-16 each).
// (Thresholds say nothing of the values' size: they may be far above it.)
// The largest value of a token, as bits that compare as it does; k from it.  (fp16 holds nothing below 2^-24.)
template <int NG>
__device__ __forceinline__ uint32_t largest_value(const uint32_t (&meta)[NG]) {
  float top = 0.0f;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const float s = __half2float(__ushort_as_half(meta[n] & 0xffff)), z = __half2float(__ushort_as_half(meta[n] >> 16));
    top = fmaxf(top, fmaxf(fabsf(z), fabsf(fmaf(3.0f, s, z))));
  }
  return __float_as_uint(top);
}
// Of two pairs {fp16 s, fp16 z} side by side, in fp16 (an infinity, which only its rounding gives, counts as fp16's last).
__device__ __forceinline__ __half2 largest_values(uint2 meta) {
  const uint32_t s = __byte_perm(meta.x, meta.y, 0x5410), z = __byte_perm(meta.x, meta.y, 0x7632);
  const __half2 z2 = *reinterpret_cast<const __half2*>(&z);
  return __hmax2(__habs2(z2), __habs2(__hfma2(__float2half2_rn(3.0f), *reinterpret_cast<const __half2*>(&s), z2)));
}
__device__ __forceinline__ int value_exponent(uint32_t largest) { return min(max(static_cast<int>(largest >> 23) - 127, -24), 15) + 9; }
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(127 + min(max(e, -126), 126)) << 23);
}
// s 2^(24 - 2 at - k) for the places at = 0 ... 4 in a word, and z 2^-k, of a token's {fp16 s, fp16 z}; down = 2^-k.
__device__ __forceinline__ void value_steps(uint32_t meta, float down, __half2 (&s)[5], __half2& z) {
  const __half2 quarter = __float2half2_rn(0.25f);
  s[0] = __float2half2_rn(__half2float(__ushort_as_half(meta & 0xffff)) * (down * 0x1p24f));
  z = __float2half2_rn(__half2float(__ushort_as_half(meta >> 16)) * down);
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
