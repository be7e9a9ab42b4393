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
constexpr float kTiny = 7.8886090522101181e-31f;  // 2^-100

// n of a channel, from x / s by one multiplication. bf16 values and scales
// have 8 significant bits, so x / s is a tie (a whole number and a half) or away
// from one by more than 2^-11 of itself; a reciprocal that is larger by 2^-20
// moves ties past the half, and nothing else across one. Adding 1.5 * 2^23
// leaves the rounded number in the low bits.
// As sign (bit 7) and magnitude.
__device__ __forceinline__ uint32_t quant_code(float x, float inv) {
  return (__float_as_uint(fmaf(fabsf(x), inv, 12582912.f)) & 0x7fu) | (__float_as_uint(x) >> 24 & 0x80u);
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
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r < lo || r >= hi) continue;  // the same for the whole warp
    const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
    // The largest magnitude, as bit patterns: those of infinities and NaN are the largest.
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float amax = __uint_as_float(top);
    __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(amax, BITS == 4 ? 7.f : 127.f));
    const float sf = __bfloat162float(s);
    float inv = __frcp_rn(sf) * (1.f + 9.5367431640625e-7f);
    if (!(amax >= kTiny)) {
      inv = 0.f;
      s = __ushort_as_bfloat16(0);
    }
    const bool bad = top >= 0x7f800000u;  // an infinity or NaN in the group: the whole group reads as NaN
    if (bad) s = __ushort_as_bfloat16(0x7fc0);
    uint32_t n[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      n[2 * e] = bad ? 0u : quant_code(bf16lo_to_f32(w[e]), inv);
      n[2 * e + 1] = bad ? 0u : quant_code(bf16hi_to_f32(w[e]), inv);
    }
    uint8_t* rec = rec0 + r * kRec;
    if ((j & 3) == 0)
      reinterpret_cast<__nv_bfloat16*>(rec + cache_scale_offset(BITS))[(is_v ? 4 : 0) + G] = s;
    auto sign = [&](int i) { return n[i] >> 7; };
    auto mag = [&](int i) { return n[i] & 0x7fu; };
    if (!is_v) {
      uint32_t* words = reinterpret_cast<uint32_t*>(rec);
      if (BITS == 4) {
        words[4 * (j & 3) + G] = pack_fields(n[0], n[2], n[4], n[6]) | pack_fields(n[1], n[3], n[5], n[7]) << 16;
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          words[16 * (G >> 1) + 4 * (j & 3) + 2 * (G & 1) + f] =
              mag(4 * f) | sign(4 * f) << 15 | mag(4 * f + 1) << 16 | sign(4 * f + 1) << 31 | mag(4 * f + 2) << 8 |
              sign(4 * f + 2) << 23 | mag(4 * f + 3) << 24 | sign(4 * f + 3) << 7;
      }
    } else {
      uint8_t* at = rec + cache_v_offset(BITS);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const int g = 2 * (j & 3) + f, i = 4 * f;
        if (BITS == 4)
          reinterpret_cast<uint16_t*>(at)[4 * g + G] =
              static_cast<uint16_t>(pack_fields(n[i], n[i + 1], n[i + 2], n[i + 3]));
        else
          reinterpret_cast<uint32_t*>(at)[4 * g + G] = n[i] | n[i + 1] << 8 | n[i + 2] << 16 | n[i + 3] << 24;
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
