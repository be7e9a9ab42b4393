// The quantised K/V cache (kv_cache.cuh): rows written from bf16 K and V, and
// read back as bf16.
//
//   s = bf16(max |x| / m),  n = x / s to the nearest, ties away from zero,
//   value n * s;  m = 7 (4 bits) or 127 (8 bits), a scale per 32 channels.
//
// Both move bytes and little else (a written row is 512 bytes in and 144 or
// 272 out, a read one the reverse), so HBM bounds them, and the launch where
// there are few rows. A warp takes kRows rows of one head: half of it K, half V,
// eight channels a lane, so that a row is one 16-byte access of every lane and
// all rows' loads are in flight at once. Neighbouring warps take neighbouring
// heads, whose rows lie side by side in K and V. Records go through shared
// memory, where a lane's codes are scattered over the row, and leave or arrive
// as contiguous 16-byte accesses: the rows of a head follow one another.
//
// 32768 tokens x 32 heads, 103 us in 4 bits and 123 in 8 at the 6.7 TB/s that a plain
// copy reaches: read back in 103 and 119, written in 107 and 120. At the memory's rate
// an SM has 116 issue slots for a written row's 256 numbers, and in 4 bits they are
// what is short: with K's and V's lanes in branches of their own, a division a group
// and signs moved one by one it took 203 us, with operands selected instead 143, with
// the sums of products below 120, and with all eight rows of a warp in one piece of
// code where they all exist 107 (92 instructions a row). 1777 tokens x 3 x 8 heads in
// 8 bits: written in 7.8 us, read in 6.7 (of 5.0 by bytes); one token: 2.1 and 1.6.
#include <cuda_bf16.h>

#include <algorithm>

#include "kv_cache.cuh"
#include "lcb_internal.h"

namespace lcb {
namespace {

constexpr int kD = 128;
constexpr int kWarps = 4;
constexpr int kRows = 8;  // rows of a warp

// A group whose largest magnitude is below this is held as zeros: the scales
// of the others, and their reciprocals, are then normal numbers.
constexpr float kTiny = 0x1p-100f;

// |n| of a channel, from |x| / s by one multiplication. bf16 values and scales
// have 8 significant bits, so x / s is a tie (a whole number and a half) or away
// from one by more than 2^-12 of itself up to 7, and 2^-16 up to 127. The reciprocal
// is off by 2^-23 of itself at most, and times 1 + 2^-20, rounded, too large by
// 2^-21 to 2^-19: ties move past the half, and nothing else across one.
// Adding 1.5 * 2^23 leaves the rounded number in the low bits of the result.
__device__ __forceinline__ uint32_t magnitude(float x, float inv) {
  return __float_as_uint(fmaf(fabsf(x), inv, 12582912.f));
}
constexpr uint32_t kMagic = 0x4b400000u;  // the bits around it

// The larger magnitudes of two pairs of bf16 (with some sign); NaN where there is one.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int BITS>
__global__ void __launch_bounds__(32 * kWarps, 8) kv_cache_write_kernel(const __grid_constant__ KvCacheWrite p) {
  constexpr int kRec = cache_row_bytes(BITS);
  __shared__ __align__(16) uint8_t recs[kWarps][kRows * kRec];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = blockIdx.x * kWarps + warp;
  if (unit >= p.units) return;
  const uint32_t bt = unit / static_cast<uint32_t>(p.Hkv);
  const int h = static_cast<int>(unit - bt * p.Hkv);
  const int b = static_cast<int>(bt / static_cast<uint32_t>(p.blocks));
  const int t0 = static_cast<int>(bt - static_cast<uint32_t>(b) * p.blocks) * kRows;
  // token t goes to row first + t
  const long long first = static_cast<long long>(p.lens[b]) - p.T;
  const int lo = static_cast<int>(max(0LL, min(static_cast<long long>(kRows), -first - t0)));
  const int hi = static_cast<int>(max(0LL, min(static_cast<long long>(min(kRows, p.T - t0)), p.Smax - first - t0)));
  if (lo >= hi) return;
  const bool is_v = lane >= 16;
  const int j = lane & 15;  // channels 8 j .. 8 j + 7
  const int G = j >> 2;
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + b * p.batch_stride + t0 * p.row_stride + h * kD + 8 * j;
  uint4 x[kRows];
  const bool full = lo == 0 && hi == kRows;
  if (full) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) x[r] = __ldcs(reinterpret_cast<const uint4*>(src + r * p.row_stride));
  } else {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r >= lo && r < hi) x[r] = __ldcs(reinterpret_cast<const uint4*>(src + r * p.row_stride));
  }
  uint8_t* rec0 = recs[warp];
  // Where in a record the lane's scale and its two pieces of codes go: K's side by side, V's those of two lanes' operands.
  const int t = j & 3;
  const int scale_at = cache_scale_offset(BITS) + 2 * ((is_v ? 4 : 0) + G);
  const int code_at = BITS == 4 ? (is_v ? 64 + 16 * t + 2 * G : 16 * t + 4 * G)
                                : (is_v ? 128 + 32 * t + 4 * G : 64 * (G >> 1) + 16 * t + 8 * (G & 1));
  const int code_step = BITS == 4 ? (is_v ? 8 : 2) : (is_v ? 16 : 4);
  // K and V differ in the order of their codes. So that all lanes do the same, a word's magnitudes are summed with the
  // lane's own powers of two (mod 2^32, where kMagic's share is taken off at the start), and its signs gathered by the
  // lane's own byte selectors. 4 bits: channel e's field is e / 2 of half e % 2 (K) or e % 4 of half e / 4 (V).
  uint32_t mul[8], base = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (BITS == 4) {
      const int i = is_v ? e & 3 : e >> 1;
      mul[e] = 1u << (16 * (is_v ? e >> 2 : e & 1) + 8 * (i >> 1) + 3 * (i & 1));
      base -= kMagic * mul[e];
    } else {
      const int i = e & 3;  // both words alike: bytes 0 2 1 3 (K), 0 1 2 3 (V)
      mul[e] = 1u << 8 * (is_v || i == 0 || i == 3 ? i : 3 - i);
      if (e < 4) base -= kMagic * mul[e];
    }
  }
  const uint32_t sel_a = is_v ? 0x7531 : 0x3715;  // 4 bits; the sign bytes of words 0, 2 and of words 1, 3
  const uint32_t sel_c = is_v ? 0x2604 : 0x3210, sel_d = is_v ? 0x3715 : 0x7654;
  const uint32_t sel_8 = is_v ? 0x7531 : 0x3517;
  auto row = [&](int r) {
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    // The largest magnitude of the group.
    uint32_t top = max_abs_bf16x2(max_abs_bf16x2(w[0], w[1]), max_abs_bf16x2(w[2], w[3]));
    top = max_abs_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_abs_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t amax_bits = max(top << 16 & 0x7fff0000u, top & 0x7fff0000u);
    // The scale. max / m times 1 / m as a number: no quotient lies so near a midpoint that it would round another way.
    const float amax = __uint_as_float(amax_bits);
    uint32_t s = __bfloat16_as_ushort(__float2bfloat16_rn(amax * (BITS == 4 ? 1.f / 7.f : 1.f / 127.f)));
    float inv = rcp_approx(__uint_as_float(s << 16)) * (1.f + 9.5367431640625e-7f);
    const bool bad = amax_bits >= 0x7f800000u;  // an infinity or NaN in the group: the whole group reads as NaN
    const bool none = !(amax >= kTiny);         // (NaN too)
    if (none) s = 0, inv = 0.f;
    if (bad) s = 0x7fc0;
    uint8_t* rec = rec0 + r * kRec;
    if ((j & 3) == 0) *reinterpret_cast<uint16_t*>(rec + scale_at) = static_cast<uint16_t>(s);
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[2 * e] = magnitude(bf16lo_to_f32(w[e]), inv);
      n[2 * e + 1] = magnitude(bf16hi_to_f32(w[e]), inv);
    }
    if (BITS == 4) {
      uint32_t sum = base;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += n[e] * mul[e];
      if (bad) sum = 0;
      const uint32_t a = permute_bytes(w[0], w[2], sel_a), c = permute_bytes(w[1], w[3], sel_a);
      const uint32_t even = permute_bytes(a, c, sel_c), odd = permute_bytes(a, c, sel_d);
      const uint32_t word = sum | ((even & 0x80808080u) | (odd >> 1 & 0x40404040u));
      *reinterpret_cast<uint16_t*>(rec + code_at) = static_cast<uint16_t>(word);
      *reinterpret_cast<uint16_t*>(rec + code_at + code_step) = static_cast<uint16_t>(word >> 16);
    } else {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        uint32_t sum = base;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += n[4 * f + e] * mul[e];
        if (bad) sum = 0;
        *reinterpret_cast<uint32_t*>(rec + code_at + f * code_step) =
            sum | (permute_bytes(w[2 * f], w[2 * f + 1], sel_8) & 0x80808080u);
      }
    }
  };
  if (full) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) row(r);
  } else {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r >= lo && r < hi) row(r);  // the same for the whole warp
  }
  __syncwarp();
  uint4* dst = reinterpret_cast<uint4*>(p.cache + b * p.cache_batch_stride + h * p.cache_head_stride +
                                        (first + t0) * kRec);
  const uint4* from = reinterpret_cast<const uint4*>(rec0);
  for (int i = lo * (kRec / 16) + lane; i < hi * (kRec / 16); i += 32) dst[i] = from[i];
}

template <int BITS>
__global__ void __launch_bounds__(32 * kWarps) kv_cache_read_kernel(const __grid_constant__ KvCacheRead p) {
  constexpr int kRec = cache_row_bytes(BITS);
  constexpr int kVecs = kRows * kRec / 16;  // 16-byte vectors of a warp's rows
  __shared__ __align__(16) uint8_t recs[kWarps][kRows * kRec];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t unit = blockIdx.x * kWarps + warp;
  if (unit >= p.units) return;
  const uint32_t bt = unit / static_cast<uint32_t>(p.Hkv);
  const int h = static_cast<int>(unit - bt * p.Hkv);
  const int b = static_cast<int>(bt / static_cast<uint32_t>(p.blocks));
  const int t0 = static_cast<int>(bt - static_cast<uint32_t>(b) * p.blocks) * kRows;
  const int rows = min(kRows, p.n - t0);
  // rows of the cache that are filled; the others read as zeros
  const int have = p.lens ? max(0, min(rows, max(p.lens[b], 0) - (p.start + t0))) : rows;
  const uint4* src = reinterpret_cast<const uint4*>(p.cache + b * p.cache_batch_stride + h * p.cache_head_stride +
                                                    static_cast<long long>(p.start + t0) * kRec);
  uint4* rec16 = reinterpret_cast<uint4*>(recs[warp]);
  uint4 x[(kVecs + 31) / 32];
#pragma unroll
  for (int i = 0; i < (kVecs + 31) / 32; ++i) {
    const int at = 32 * i + lane;
    if (at < have * (kRec / 16)) x[i] = __ldcs(src + at);
  }
#pragma unroll
  for (int i = 0; i < (kVecs + 31) / 32; ++i) {
    const int at = 32 * i + lane;
    if (at < have * (kRec / 16)) rec16[at] = x[i];
  }
  __syncwarp();
  const bool is_v = lane >= 16;
  const int j = lane & 15, G = j >> 2;  // channels 8 j .. 8 j + 7
  __nv_bfloat16* dst = (is_v ? p.v : p.k) + b * p.batch_stride + t0 * p.row_stride + h * kD + 8 * j;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r >= rows) break;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (r < have) {
      const uint8_t* rec = recs[warp] + r * kRec;
      const uint32_t s1 = reinterpret_cast<const uint16_t*>(rec + cache_scale_offset(BITS))[(is_v ? 4 : 0) + G];
      const uint32_t s = s1 | s1 << 16;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(rec);
      if (!is_v && BITS == 4) {
        const Fields x = k4_fields(words[4 * (j & 3) + G]);
#pragma unroll
        for (int f = 0; f < 4; ++f) w[f] = f & 1 ? (x.pair(f) & 0x80008000u) | (x.pair(f) >> 4 & 0x00070007u) : x.pair(f);
      } else if (!is_v) {
        const uint32_t* two = words + 16 * (G >> 1) + 4 * (j & 3) + 2 * (G & 1);
#pragma unroll
        for (int f = 0; f < 4; ++f) w[f] = k8_f16x2(two[f >> 1], f & 1);
      } else if (BITS == 4) {
        const uint16_t* half = reinterpret_cast<const uint16_t*>(rec + cache_v_offset(BITS));
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t a = half[4 * (2 * (j & 3) + f) + G];
          // fields 0, 1 and 2, 3 as pairs
          w[2 * f] = (a & 0x8007u) | (a << 13 & 0x70000u) | (a << 17 & 0x80000000u);
          w[2 * f + 1] = (a >> 8 & 7u) | (a << 8 & 0x8000u) | (a << 5 & 0x70000u) | (a << 25 & 0x80000000u);
        }
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t x = words[cache_v_offset(BITS) / 4 + 4 * (2 * (j & 3) + f) + G];
          w[2 * f] = permute_bytes(x, 0, 0x9180);
          w[2 * f + 1] = permute_bytes(x, 0, 0xb3a2);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = signed_bf16x2(w[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = hmul2_bf16(w[e], s);  // the one rounding: n and s have 8 bits each
    }
    __stcs(reinterpret_cast<uint4*>(dst + r * p.row_stride), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// Warps' units of B sequences of n rows and Hkv heads; below zero where there are more than 32 bits number (2^35 rows).
long long units_of(int B, int n, int Hkv, int& blocks) {
  blocks = n / kRows + (n % kRows != 0);
  const long long rows = static_cast<long long>(B) * blocks;
  if (rows == 0) return 0;
  return rows > 0xffffffffLL / Hkv ? -1 : rows * Hkv;
}

}  // namespace

int launch_kv_cache_write(KvCacheWrite p, int bits, cudaStream_t stream) {
  const long long units = units_of(p.B, p.T, p.Hkv, p.blocks);
  if (units < 0) return -1;
  if (units == 0) return 0;
  p.units = static_cast<unsigned>(units);
  const unsigned grid = p.units / kWarps + (p.units % kWarps != 0);
  if (bits == 4)
    kv_cache_write_kernel<4><<<grid, 32 * kWarps, 0, stream>>>(p);
  else
    kv_cache_write_kernel<8><<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_kv_cache_read(KvCacheRead p, int bits, cudaStream_t stream) {
  const long long units = units_of(p.B, p.n, p.Hkv, p.blocks);
  if (units < 0) return -1;
  if (units == 0) return 0;
  p.units = static_cast<unsigned>(units);
  const unsigned grid = p.units / kWarps + (p.units % kWarps != 0);
  if (bits == 4)
    kv_cache_read_kernel<4><<<grid, 32 * kWarps, 0, stream>>>(p);
  else
    kv_cache_read_kernel<8><<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
