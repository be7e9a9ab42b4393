// The quantised K/V cache: how a cached row of a K/V head lies in memory.
//
// A row holds a K and a V vector of 128 channels. Each group of 32 channels
// has a bf16 scale s; channel c holds s * n with a whole number n: -7 .. 7 in a
// 4-bit cache, -127 .. 127 in an 8-bit one, kept as a sign and a magnitude. The
// row is one record of
//   16 * bits bytes   K codes
//   16 * bits bytes   V codes
//   8 + 8 bytes       K's and V's four scales
// (144 bytes in 4 bits, 272 in 8), so that one contiguous stream carries all
// that attention reads of a head.
//
// The codes lie as a lane (g, t) of a warp takes them for operands of tensor
// products (the sum over channels and the order of O's channels are free to
// permute). A magnitude in the low bits of a floating-point number whose
// exponent is zero is a subnormal number, a power of two times the magnitude,
// and tensor cores multiply those exactly; so one bitwise AND, after at most a
// rotation, a byte permute and a shift, takes a pair of codes:
//   4 bits: four codes in 16 bits, as fields 0 .. 3. ANDed with 0x8007 they
//     leave field 0; shifted left by 1 and ANDed with 0x8070 field 1, 2^4 as
//     large; with the two bytes exchanged before, fields 2 and 3.
//   K, 4 bits: lane t takes channels 32 G + 8 t .. + 7 of the groups G = 0 .. 3,
//     word 4 t + G, as pairs of fp16: field i of its halves has channels 2 i and
//     2 i + 1 (n * 2^-24 or n * 2^-20).
//   K, 8 bits: the same channels, words 16 (G / 2) + 4 t + 2 (G % 2) + {0, 1}, as
//     fp16 (n * 2^-24). A word ANDed with 0x807f807f has the first two of its four
//     channels, rotated right by 8 bits before that the others.
//   V, 4 bits: lane g takes channels 32 G + 4 g .. + 3 of each group, half-word
//     4 g + G, its fields. Those of two keys side by side in a register are pairs
//     of bf16 (n * 2^-133 or n * 2^-129).
//   V, 8 bits: the same channels, bytes 16 g + 4 G + {0 .. 3}, sign and magnitude:
//     a byte permute that repeats the sign, ANDed with 0x807f807f, makes those of
//     two keys a bf16 pair (n * 2^-133).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace lcb {

constexpr int cache_v_offset(int bits) { return 16 * bits; }
constexpr int cache_scale_offset(int bits) { return 32 * bits; }
constexpr int cache_row_bytes(int bits) { return 32 * bits + 16; }

// Bytes of (a, b) by the nibbles of `sel`, the highest bit of a nibble giving eight copies of that byte's sign.
__device__ __forceinline__ uint32_t permute_bytes(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t rotate_right(uint32_t x, int n) { return __funnelshift_r(x, x, n); }

// Fields of both halves of a word.
struct Fields {
  uint32_t x, y;  // the word, and with the bytes of its halves exchanged
  __device__ __forceinline__ uint32_t pair(int i) const {
    const uint32_t v = i < 2 ? x : y;
    return i & 1 ? (v << 1) & 0x80708070u : v & 0x80078007u;
  }
};

// K of a lane's word in 4 bits, as pairs of fp16.
__device__ __forceinline__ Fields k4_fields(uint32_t w) { return {w, permute_bytes(w, w, 0x2301)}; }

// V of one channel group of two keys in 4 bits, from the words that have it (G odd: in the high half), as pairs of bf16.
__device__ __forceinline__ Fields v4_fields(uint32_t key0, uint32_t key1, int G) {
  return {permute_bytes(key0, key1, G & 1 ? 0x7632 : 0x5410), permute_bytes(key0, key1, G & 1 ? 0x6723 : 0x4501)};
}

// K of a word in 8 bits: channels 2 f and 2 f + 1 of its four, as fp16.
__device__ __forceinline__ uint32_t k8_f16x2(uint32_t w, int f) { return (f ? rotate_right(w, 8) : w) & 0x807f807fu; }

// V of one channel group of two keys in 8 bits.
struct V8 {
  uint32_t key0, key1;
  __device__ __forceinline__ uint32_t pair(int i) const {
    return permute_bytes(key0, key1, 0xc480u + 0x1111u * static_cast<uint32_t>(i)) & 0x807f807fu;
  }
};

// A word of signs and magnitudes, sign and 7 bits at each end of 16, as whole numbers in bf16. Exact.
__device__ __forceinline__ uint32_t signed_bf16x2(uint32_t x) {
  uint32_t r;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((x & 0x007f007fu) | 0x43004300u), "r"(0xc300c300u));  // 128 + u - 128
  return r | (x & 0x80008000u);
}

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

}  // namespace lcb
