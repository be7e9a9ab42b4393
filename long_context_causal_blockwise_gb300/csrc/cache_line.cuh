// Attention over the quantised cache (attn_cache_decode.cu, attn_cache_tiles.cu):
// the keys that a tile of query rows sees, and their deal over the GPU.
#pragma once

#include "attn_window.cuh"
#include "kv_cache.cuh"
#include "lcb_internal.h"
#include "mma_warp.cuh"

namespace lcb {

constexpr int kCacheD = 128;
constexpr int kLineSequences = 1024;  // whose lengths a CTA keeps in shared memory
constexpr int kQTop = 15;  // a row's largest element of Q goes to [2^15, 2^16) in fp16: bf16's largest mantissa fits
constexpr float kLeastFactor = 0x1p-149f;  // of a score: fp32's smallest number

// Rows of a sequence in the cache.
__device__ __forceinline__ int length(const CacheDecode& p, int len) { return min(max(len, 0), p.Smax); }

// A row tile of a (sequence, K/V head), and the keys that a row of it sees:
// [0, ns) and [lo, hi), in units of `keys` that do not cross from one to the
// other; every key of the units [whole0, whole1) is seen by every row.
struct Tile {
  int b, hk, r0;         // rows r = (token r / G, query head hk * G + r % G), r0 <= r < r0 + rows
  int p0, p_min, p_max;  // positions of token 0, of the tile's first row and of its last
  int lo, hi, ns, sink_units, units, whole0, whole1;
};

__device__ __forceinline__ Tile make_tile(const CacheDecode& p, int len, int b, int hk, int mt, int rows,
                                          int keys) {
  Tile a;
  a.b = b;
  a.hk = hk;
  a.r0 = mt * rows;
  a.p0 = len - p.T;
  a.p_min = a.p0;
  a.p_max = len - 1;
  if (p.row_tiles > 1) {
    a.p_min = a.p0 + a.r0 / p.G;
    a.p_max = a.p0 + min(p.T * p.G - 1, a.r0 + rows - 1) / p.G;
  }
  a.lo = max(0, a.p_min - p.window + 1);
  a.hi = max(a.lo, a.p_max + 1);
  a.ns = max(0, min(min(p.sinks, a.lo), a.p_max + 1));
  a.sink_units = (a.ns + keys - 1) / keys;
  a.units = a.sink_units + (a.hi - a.lo + keys - 1) / keys;
  a.whole0 = a.sink_units + (max(0, a.p_max - p.window + 1 - a.lo) + keys - 1) / keys;
  a.whole1 = a.sink_units + max(0, min(a.p_min + 1, a.hi) - a.lo) / keys;
  return a;
}

__device__ __forceinline__ int first_key(const Tile& a, int u, int keys) {
  return u * keys + (u < a.sink_units ? 0 : a.lo - a.sink_units * keys);
}
// Keys of unit u, whose first is j0.
__device__ __forceinline__ int keys_of(const Tile& a, int u, int j0, int keys) {
  return min(keys, (u < a.sink_units ? a.ns : a.hi) - j0);
}

// n things dealt in order to `parts`, the first n % parts of which get one more.
struct Share {
  int each, more;
  __device__ Share(int n, int parts) : each(n / parts), more(n - n / parts * parts) {}
  __device__ int begin(int i) const { return i * each + min(i, more); }  // of part i
  __device__ int part_of(int x) const {                                  // that has thing x
    const int cut = more * (each + 1);
    return x < cut ? x / (each + 1) : more + (x - cut) / each;
  }
};

// Row r of a tile, four channels a lane.
__device__ __forceinline__ void store_row(const CacheDecode& p, const Tile& a, int r, float M, float L, float4 v,
                                          int lane) {
  r += a.r0;
  if (r >= p.T * p.G) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int tok = p.G == 1 ? r : r / p.G, h = a.hk * p.G + r - tok * p.G;
  uint2 x;
  x.x = pack_bf16x2(v.x * inv, v.y * inv);
  x.y = pack_bf16x2(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(p.o + a.b * p.o_bs + static_cast<long long>(tok) * p.o_rs + h * kCacheD + 4 * lane) = x;
  if (lane == 0) p.lse[a.b * p.l_bs + h * p.l_hs + tok] = L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ the units of all tiles as one line
//
// Tiles stand in the order (sequence, K/V head, row tile), each with as many
// places as it has units, and kTileCost more in front of those where it has any:
// what a CTA spends on coming to another tile (its last one's sums stored, Q, an
// empty pipeline), in units. The N places (fewer than 2^31) are dealt in order to
// C CTAs, C at most N. What a CTA has of a tile that it does not have whole goes
// to slot 2 i (the first tile of which it has a unit) or 2 i + 1 (the last): ROWS
// x 128 sums, then the rows' maxima, then their sums of weights.
// (us, without the cost / with it: 8 tiles of 512 units with 128 rows, of which 7
// of 152 CTAs see two, 55 / 48; 8 heads x 65536 keys, eight rows 30 / 26; 4 x 100000,
// six rows, 26.5 / 23.4; 8 x 524288, four rows, 104 / 103. Half or one
// and a half times the cost: within 2% for four and eight rows, 5% for the others.)

template <int ROWS>
constexpr int kTileCost = ROWS == 128 ? 7 : ROWS == 16 ? 9 : ROWS == 8 ? 5 : 4;
template <int ROWS>
__device__ __forceinline__ int places(int units) { return units > 0 ? units + kTileCost<ROWS> : 0; }

constexpr int slot_floats(int rows) { return rows * (kCacheD + 2); }

// Places of the first n row tiles of a K/V head.
template <int ROWS>
__device__ __forceinline__ int head_places(const CacheDecode& p, int len, int n, int keys) {
  int x = 0;
  for (int mt = 0; mt < n; ++mt) x += places<ROWS>(make_tile(p, len, 0, 0, mt, ROWS, keys).units);
  return x;
}
// The same by a whole warp.
template <int ROWS>
__device__ __forceinline__ int head_places_warp(const CacheDecode& p, int len, int n, int keys, int lane) {
  int x = 0;
  for (int mt = lane; mt < n; mt += 32) x += places<ROWS>(make_tile(p, len, 0, 0, mt, ROWS, keys).units);
  return __reduce_add_sync(0xffffffffu, x);
}
// Whether a warp takes the sequences one by one, its lanes the row tiles, or a lane a sequence.
__device__ __forceinline__ bool lanes_take_tiles(const CacheDecode& p) { return p.row_tiles >= 32; }

// The places of all sequences, and of those before `b`, by a whole warp. (lens may be the caller's own: lengths past the
// cache, or below zero, count as they do everywhere.)
template <int ROWS>
__device__ __forceinline__ int all_places(const CacheDecode& p, const int* lens, int b, int keys, int lane, int* before) {
  int n = 0, m = 0;
  if (lanes_take_tiles(p)) {
    for (int i = 0; i < p.B; ++i) {
      if (i == b) m = n;
      n += p.Hkv * head_places_warp<ROWS>(p, length(p, lens[i]), p.row_tiles, keys, lane);
    }
    *before = m;
    return n;
  }
  for (int i = lane; i < p.B; i += 32) {
    const int x = p.Hkv * head_places<ROWS>(p, length(p, lens[i]), p.row_tiles, keys);
    n += x;
    if (i < b) m += x;
  }
  *before = __reduce_add_sync(0xffffffffu, m);
  return __reduce_add_sync(0xffffffffu, n);
}

// The sequence of place x, and the places before it.
template <int ROWS>
__device__ __forceinline__ int sequence_of(const CacheDecode& p, const int* lens, int x, int keys, int lane, int* before) {
  int sum = 0;
  if (lanes_take_tiles(p)) {
    for (int b = 0;; ++b) {
      const int next = sum + p.Hkv * head_places_warp<ROWS>(p, lens[b], p.row_tiles, keys, lane);
      if (next > x || b == p.B - 1) {
        *before = sum;
        return b;
      }
      sum = next;
    }
  }
  for (int b0 = 0;; b0 += 32) {
    const int mine = b0 + lane < p.B ? p.Hkv * head_places<ROWS>(p, lens[b0 + lane], p.row_tiles, keys) : 0;
    int upto = mine;  // inclusive prefix
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, sum + upto > x);
    if (past || b0 + 32 >= p.B) {
      const int i = past ? __ffs(past) - 1 : 31;
      *before = sum + __shfl_sync(0xffffffffu, upto - mine, i);
      return min(b0 + i, p.B - 1);
    }
    sum += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// A CTA's way along the line. The lengths are a copy that the CTA made (one for
// all its warps, which otherwise might disagree about it if somebody changes
// them meanwhile, and wait for one another for ever).
template <int ROWS, int KEYS>
struct Walk {
  Tile a;
  int off, left;  // the CTA's next unit in the tile; places that it still has
  int b, hk, mt;

  // False for a CTA without units.
  __device__ __forceinline__ bool start(const CacheDecode& p, const int* lens, int cta, int ctas, int lane) {
    int before;
    const int N = all_places<ROWS>(p, lens, 0, KEYS, lane, &before);
    const int C = min(N, ctas);
    if (cta >= C) return false;
    const Share share(N, C);
    int x = share.begin(cta);
    left = share.begin(cta + 1) - x;
    b = sequence_of<ROWS>(p, lens, x, KEYS, lane, &before);
    const int per_head = head_places_warp<ROWS>(p, lens[b], p.row_tiles, KEYS, lane);
    x -= before;
    hk = x / per_head;
    x -= hk * per_head;
    for (mt = 0;; ++mt) {
      a = make_tile(p, lens[b], b, hk, mt, ROWS, KEYS);
      if (x < places<ROWS>(a.units) || mt == p.row_tiles - 1) break;
      x -= places<ROWS>(a.units);
    }
    off = max(0, x - kTileCost<ROWS>);
    left -= max(0, kTileCost<ROWS> - x);
    return left > 0;
  }
  // Units of the present tile that are the CTA's.
  __device__ __forceinline__ int here() const { return min(left, a.units - off); }
  __device__ __forceinline__ void advance(const CacheDecode& p, const int* lens, int n) {
    left -= n;
    off += n;
    while (off >= a.units && left > 0) {
      off = 0;
      if (++mt == p.row_tiles) {
        mt = 0;
        if (++hk == p.Hkv) {
          hk = 0;
          if (++b == p.B) left = b = 0;
        }
      }
      a = make_tile(p, lens[b], b, hk, mt, ROWS, KEYS);
      if (a.units > 0) left -= kTileCost<ROWS>;
    }
  }
};

// A CTA's copy of the lengths.
__device__ __forceinline__ void copy_lengths(const CacheDecode& p, int* lens) {
  for (int i = threadIdx.x; i < p.B; i += blockDim.x) lens[i] = length(p, p.lens[i]);
}

// kSplit warps join a row of a tile that several CTAs share; rows of tiles
// without a key get their zeros here.
template <int ROWS, int KEYS, int kSplit>
__global__ void __launch_bounds__(256) cache_decode_join_kernel(const __grid_constant__ CacheDecode p, int ctas,
                                                                int blocks) {
  constexpr int kSlot = slot_floats(ROWS);
  constexpr int kRowsHere = 8 / kSplit;
  __shared__ float4 sO[8][32];
  __shared__ float sM[8], sL[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int tile = static_cast<int>(blockIdx.x) / blocks;  // of which a tile has so many
  const int sub = static_cast<int>(blockIdx.x) - tile * blocks;
  const int mt = tile % p.row_tiles;
  tile /= p.row_tiles;
  const int b = tile / p.Hkv, hk = tile % p.Hkv;
  const int len = length(p, p.lens[b]);
  const Tile a = make_tile(p, len, b, hk, mt, ROWS, KEYS);
  int start;  // the tile's first place
  const int N = all_places<ROWS>(p, p.lens, b, KEYS, lane, &start);
  start += hk * head_places_warp<ROWS>(p, len, p.row_tiles, KEYS, lane) + head_places_warp<ROWS>(p, len, mt, KEYS, lane);
  const int r = sub * kRowsHere + warp / kSplit, part = warp % kSplit;
  const Share share(max(N, 1), max(1, min(N, ctas)));
  // the CTAs of its first and last units (never past the slots that there are, even if somebody changes the lengths
  // meanwhile), and whether the first one has none of the tile before
  const int unit0 = start + kTileCost<ROWS>;
  const int i0 = min(share.part_of(unit0), ctas - 1), i1 = min(share.part_of(unit0 + max(a.units, 1) - 1), ctas - 1);
  const bool at_start = share.begin(i0) >= start;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.r0 + r >= p.T * p.G) {  // the last tile has fewer rows
    if (kSplit > 1 && kRowsHere > 1) __syncthreads();
    return;
  }
  if (a.units == 0) {
    if (part == 0) store_row(p, a, r, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f), lane);
    return;
  }
  if (i0 == i1) return;  // stored by the one CTA that has it
  float M = -INFINITY, L = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = i0 + part; i <= i1; i += kSplit) {
    const float* slot = p.workspace + (2LL * i + (i > i0 || at_start ? 0 : 1)) * kSlot;
    const float4 y = *reinterpret_cast<const float4*>(slot + r * kCacheD + 4 * lane);
    const float m = slot[ROWS * kCacheD + r], l = slot[ROWS * (kCacheD + 1) + r];
    const float top = fmaxf(M, m), f = weight(M, top), g = weight(m, top);
    M = top;
    L = f * L + g * l;
    v = make_float4(f * v.x + g * y.x, f * v.y + g * y.y, f * v.z + g * y.z, f * v.w + g * y.w);
  }
  if (kSplit > 1) {
    sO[warp][lane] = v;
    if (lane == 0) {
      sM[warp] = M;
      sL[warp] = L;
    }
    __syncthreads();
    if (part != 0) return;
    float top = M;
#pragma unroll
    for (int i = 1; i < kSplit; ++i) top = fmaxf(top, sM[warp + i]);
    const float f = weight(M, top);
    M = top;
    L *= f;
    v = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
#pragma unroll
    for (int i = 1; i < kSplit; ++i) {
      const float4 x = sO[warp + i][lane];
      const float g = weight(sM[warp + i], top);
      L += g * sL[warp + i];
      v = make_float4(v.x + g * x.x, v.y + g * x.y, v.z + g * x.z, v.w + g * x.w);
    }
  }
  store_row(p, a, r, M, L, v, lane);
}

// The join after a line kernel of n CTAs, which may start beside its end.
template <int ROWS, int KEYS>
int launch_cache_join(const CacheDecode& p, long long tiles, int n, cudaStream_t stream) {
  // A warp or two a row where a tile has few parts, eight where it has many.
  constexpr int kNarrow = ROWS == 4 ? 2 : 1;
  const bool wide = n > 8 * tiles;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int rows = p.row_tiles > 1 ? ROWS : p.T * p.G;  // of a tile
  const int blocks = wide ? rows : (rows * kNarrow + 7) / 8;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, cache_decode_join_kernel<ROWS, KEYS, 8>, p, n, blocks)
                             : cudaLaunchKernelEx(&cfg, cache_decode_join_kernel<ROWS, KEYS, kNarrow>, p, n,
                                                  blocks);
  return e == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
