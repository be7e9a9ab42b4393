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
// from one by more than 2^-11 of itself; a reciprocal that is larger by 2^-20
// moves ties past the half, and nothing else across one, its own error included.
// Adding 1.5 * 2^23 leaves the rounded number in the low bits of the result.
__device__ __forceinline__ uint32_t magnitude(float x, float inv) {
  return __float_as_uint(fmaf(fabsf(x), inv, 12582912.f));
}
constexpr uint32_t kMagic = 0x4b400000u;  // the bits around it

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four codes in 16 bits (kv_cache.cuh): magnitudes m0 .. m3 with kMagic around them; the signs are those of bytes a1, b1
// (fields 0, 2) and, by `sel`, of c and d (fields 1, 3).
__device__ __forceinline__ uint32_t pack_fields(uint32_t m0, uint32_t m1, uint32_t m2, uint32_t m3, uint32_t a, uint32_t b,
                                                uint32_t sel_ab, uint32_t c, uint32_t d, uint32_t sel_cd) {
  const uint32_t even = permute_bytes(b, a, sel_ab) & 0x8080u, odd = permute_bytes(d, c, sel_cd) & 0x8080u;
  return (m0 + 8u * m1 + 256u * m2 + 2048u * m3) & 0x3f3fu | even | odd >> 1;
}

template <int BITS>
__global__ void __launch_bounds__(32 * kWarps) kv_cache_write_kernel(const __grid_constant__ KvCacheWrite p) {
  constexpr int kRec = cache_row_bytes(BITS);
  __shared__ __align__(16) uint8_t recs[kWarps][kRows * kRec];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (unit >= p.units) return;
  const int h = static_cast<int>(unit % p.Hkv);
  const long long bt = unit / p.Hkv;
  const int t0 = static_cast<int>(bt % p.blocks) * kRows, b = static_cast<int>(bt / p.blocks);
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
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (r >= lo && r < hi) x[r] = __ldcs(reinterpret_cast<const uint4*>(src + r * p.row_stride));
  uint8_t* rec0 = recs[warp];
  // where in a record the lane's scale and its two pieces of codes go: K's side by side, V's those of two lanes' operands
  const int t = j & 3;
  const int scale_at = cache_scale_offset(BITS) + 2 * ((is_v ? 4 : 0) + G);
  const int code_at = BITS == 4 ? (is_v ? 64 + 16 * t + 2 * G : 16 * t + 4 * G)
                                : (is_v ? 128 + 32 * t + 4 * G : 64 * (G >> 1) + 16 * t + 8 * (G & 1));
  const int code_step = BITS == 4 ? (is_v ? 8 : 2) : (is_v ? 16 : 4);
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r < lo || r >= hi) continue;  // the same for the whole warp
    uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    // The largest magnitude, as bit patterns: those of infinities and NaN are the largest.
    uint32_t top = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                             max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = max(top & 0xffffu, top >> 16);
    // The scale. max / m times 1 / m as a number: no quotient lies so near a midpoint that it would round another way.
    const float amax = __uint_as_float(top << 16);
    __nv_bfloat16 s = __float2bfloat16_rn(amax * (BITS == 4 ? 1.f / 7.f : 1.f / 127.f));
    float inv = rcp_approx(__bfloat162float(s)) * (1.f + 9.5367431640625e-7f);
    const bool bad = top >= 0x7f80u;  // an infinity or NaN in the group: the whole group reads as NaN
    if (bad || amax < kTiny) {
      s = __ushort_as_bfloat16(bad ? 0x7fc0 : 0);
      inv = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] &= 0x80008000u;  // (0 times an infinity is none)
    }
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[2 * e] = magnitude(bf16lo_to_f32(w[e]), inv);
      n[2 * e + 1] = magnitude(bf16hi_to_f32(w[e]), inv);
    }
    uint8_t* rec = rec0 + r * kRec;
    if ((j & 3) == 0) *reinterpret_cast<__nv_bfloat16*>(rec + scale_at) = s;
    // K and V differ in the order of their codes: operands are chosen, so that all lanes do the same.
    if (BITS == 4) {
      // K: channels 0, 2, 4, 6 and 1, 3, 5, 7; V: 0 .. 3 and 4 .. 7
      const uint32_t n1 = is_v ? n[1] : n[2], n2 = is_v ? n[2] : n[4], n3 = is_v ? n[3] : n[6];
      const uint32_t n4 = is_v ? n[4] : n[1], n5 = is_v ? n[5] : n[3], n6 = is_v ? n[6] : n[5];
      const uint32_t lo = pack_fields(n[0], n1, n2, n3, w[0], is_v ? w[1] : w[2], 0x51, is_v ? w[0] : w[1],
                                      is_v ? w[1] : w[3], is_v ? 0x73 : 0x51);
      const uint32_t hi = pack_fields(n4, n5, n6, n[7], is_v ? w[2] : w[0], is_v ? w[3] : w[2], is_v ? 0x51 : 0x73,
                                      is_v ? w[2] : w[1], w[3], 0x73);
      *reinterpret_cast<uint16_t*>(rec + code_at) = static_cast<uint16_t>(lo);
      *reinterpret_cast<uint16_t*>(rec + code_at + code_step) = static_cast<uint16_t>(hi);
    } else {
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint32_t a = w[2 * f], c = w[2 * f + 1];
        const uint32_t n1 = is_v ? n[4 * f + 2] : n[4 * f + 1], n2 = is_v ? n[4 * f + 1] : n[4 * f + 2];
        // magnitudes of channels 0, n2, n1, 3 in bytes 0 .. 3, what is around them taken off
        const uint32_t mags = n[4 * f] + (n2 << 8) + (n1 << 16) + (n[4 * f + 3] << 24) - (kMagic + (kMagic << 8));
        const uint32_t sa = a & 0x80008000u, sc = c & 0x80008000u;
        const uint32_t signs = is_v ? permute_bytes(sa, sc, 0x7531) : sa | rotate_right(sc, 24);
        *reinterpret_cast<uint32_t*>(rec + code_at + f * code_step) = mags | signs;
      }
    }
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
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (unit >= p.units) return;
  const int h = static_cast<int>(unit % p.Hkv);
  const long long bt = unit / p.Hkv;
  const int t0 = static_cast<int>(bt % p.blocks) * kRows, b = static_cast<int>(bt / p.blocks);
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

}  // namespace

int launch_kv_cache_write(KvCacheWrite p, int bits, cudaStream_t stream) {
  p.blocks = (p.T + kRows - 1) / kRows;
  p.units = static_cast<long long>(p.B) * p.blocks * p.Hkv;
  const long long grid = (p.units + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return -1;
  if (grid == 0) return 0;
  if (bits == 4)
    kv_cache_write_kernel<4><<<static_cast<unsigned>(grid), 32 * kWarps, 0, stream>>>(p);
  else
    kv_cache_write_kernel<8><<<static_cast<unsigned>(grid), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_kv_cache_read(KvCacheRead p, int bits, cudaStream_t stream) {
  p.blocks = (p.n + kRows - 1) / kRows;
  p.units = static_cast<long long>(p.B) * p.blocks * p.Hkv;
  const long long grid = (p.units + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffLL) return -1;
  if (grid == 0) return 0;
  if (bits == 4)
    kv_cache_read_kernel<4><<<static_cast<unsigned>(grid), 32 * kWarps, 0, stream>>>(p);
  else
    kv_cache_read_kernel<8><<<static_cast<unsigned>(grid), 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
