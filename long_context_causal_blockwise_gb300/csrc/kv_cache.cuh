// The quantised K/V cache: how a cached row of a K/V head lies in memory.
//
// A row holds a K and a V vector of 128 channels. Each group of 32 channels
// has a bf16 scale s; channel c holds s * n with a whole number n: -7 .. 7 in a
// 4-bit cache, -127 .. 127 in an 8-bit one. The row is one record of
//   planes * 64 bytes   K codes
//   planes * 64 bytes   V codes
//   8 + 8 bytes         K's and V's four scales
// (144 bytes in 4 bits, 272 in 8), so that one contiguous stream carries all
// that attention reads of a head. Codes are kept off zero: u = n + 8 in one
// plane of 4-bit numbers, or u = n + 128 as two, its high and its low half.
//
// Within a plane the codes lie in the order in which a lane (g, t) of a warp
// takes them as operands of m16n8k16 products (the sum over channels and the
// order of O's channels are free to permute):
//   K: lane t takes channels 32 G + 8 t .. + 7 of the groups G = 0 .. 3, one
//      32-bit word each: word 4 t + G. Pair e of a word's channels (2e, 2e + 1)
//      is its nibbles e and e + 4, 16 bits apart, so one shift and one bitwise
//      operation make it a pair of bf16 numbers (below).
//   V: lane g takes channels 32 G + 4 g .. + 3 of each group, 16 bits each:
//      half-word 4 g + G, channel i in nibble i.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace lcb {

constexpr int kCacheGroup = 32;  // channels of a scale
constexpr int kPlaneBytes = 64;

constexpr int cache_planes(int bits) { return bits / 4; }
constexpr int cache_v_offset(int bits) { return cache_planes(bits) * kPlaneBytes; }
constexpr int cache_scale_offset(int bits) { return 2 * cache_planes(bits) * kPlaneBytes; }
constexpr int cache_row_bytes(int bits) { return cache_scale_offset(bits) + 16; }

__device__ __forceinline__ uint32_t hadd2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Nibbles 0 and 4 of x as bf16 numbers 128 + u: they become the low mantissa bits of 128.
__device__ __forceinline__ uint32_t nibbles_bf16x2(uint32_t x) { return (x & 0x000f000fu) | 0x43004300u; }

// The numbers n of nibbles i and i + 4 of a plane's word (4 bits), or of the
// high and the low plane's (8 bits), as a pair of bf16. Exact at every step:
// all are whole numbers of at most 8 significant bits.
template <int BITS>
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t w0, uint32_t w1, int i) {
  const uint32_t h = nibbles_bf16x2(w0 >> (4 * i));
  if (BITS == 4) return hadd2_bf16(h, 0xc308c308u);                 // 128 + u - 136
  const uint32_t x = hfma2_bf16(h, 0x41804180u, 0xc510c510u);       // 16 (128 + hi) - 2304 = 16 hi - 256
  return hadd2_bf16(x, nibbles_bf16x2(w1 >> (4 * i)));              // + 128 + lo: n = 16 hi + lo - 128
}

}  // namespace lcb
