// Attention over the quantised K/V cache (kv_cache.cuh) for many query rows to
// a K/V head: drafted tokens, or a chunk of a prompt, times the heads of a group.
//
// Above sixteen rows the cache's bytes are no longer what costs: unpacking them
// is, which attn_cache_decode.cu does once for every sixteen rows, and the
// products, which it issues from registers. Here a tile of 128 rows has them
// unpacked once, into shared memory in the layout of the fifth generation's
// tensor cores, and 128 x 128 x 128 products from there, scores and sums in
// tensor memory:
//
//   S_t = Q K^T (fp16), O_t += P_t V (bf16), t = 0, 1 for even and odd units of
//   128 keys: two streams with maxima and sums of their own, so that one's
//   products run while the other's weights are formed.
//
//   warps 0-3, 4-7   softmax of streams 0 and 1 (thread = query row = TMEM lane)
//   warps 8-15       unpack: 16 keys of a unit each, K, then V
//   warp 16          issues the products (all lanes walk, one elected issues)
//   warp 17          brings records, 128 keys (4 bits) or 64 (8 bits) at a time
//
// A pair of codes as they lie is a pair of subnormal numbers (kv_cache.cuh), which
// one packed multiplication by a scale times the inverse of that smallness makes
// normal. K goes to fp16 as s n over a power of two, which the scores get back. In 4
// bits s n has 3 and 8 bits, fp16's eleven. In 8 bits it is two numbers, the
// magnitude's upper 3 bits (so as exact) and its lower 4 (off by half a step, 2^-12 of
// them, 2^-15 of the largest magnitude), and two products. What is left is fp16's
// range. Sixteen keys share the power of two where the exponents of their scales,
// zeros aside, span 8 at most: s n is a multiple of 2^-24 then, and no bit is lost.
// Otherwise each key has its own, and two multiplications leave it more room: nothing
// is lost while a key's own scales span 23 (past that, a channel is off by 2^-31 of
// the key's largest scale, or twice that in 8 bits). A power of two changes no bit of
// a score, so that none depends on which keys are neighbours. Q as in
// attn_cache_decode.cu.
//
// V and the weights P are of one type, for each sixteen keys (a product's step) on
// its own. Where the sixteen keys' scales of V are ordinary (2^-7, in 8 bits 2^-11,
// up to 16, or zero) they are fp16: 2^-12 s n, off by 2^-13 of the group's largest
// value at best, 2^-9 of it at the smallest scales, and 2^7 P, off by 2^-12 down to
// weights of 2^-21 of the largest. Otherwise, and where some row of the tile does not
// see all sixteen (so that no row's bits depend on V that it does not see), bf16 with
// the same powers of two: off by half a step, 2^-9 to 2^-8 of each value. (bf16 for
// all of them: errors 2.8e-3 of the outputs instead of 1.7e-3, which is what rounding
// these to bf16 costs, and 2 us of 53 less.) NaN of V are zeros in the tile, so that
// a weight of zero leaves nothing of them; the rows that see one are told by bits, 1
// us of 53.
//
// The units of all tiles are dealt evenly to the CTAs, one to an SM, and joined
// by a second kernel (cache_line.cuh). Streams are joined first, in tensor memory:
// the warps of both see the same lanes, and take half of the channels each.
//
// Bound: 128 keys (a unit) take some 2650 clocks. Their two products take the tensor
// core 1024 of them (a tile has 128 rows whether it uses them or not), 128 rows'
// weights the exponential unit 1024, HBM 770 in 4 bits. Shared memory has the most
// to do: 96 KB that the products read, 82 KB that unpacking reads and writes, 18 KB
// that arrive, 1540 clocks at 128 bytes each; and an unpacking warp's turn (its
// sixteen keys of K 960 clocks, of V 700, two fences 330, and its waits, when a unit
// took 2440) leaves no room. 8 heads x 65536 keys, 64 rows: 50 us in 4 bits, 62 in 8;
// 32 heads x 20000, 128 rows: 59. (47, 58 and 56 before keys could have powers of two
// of their own, factors were kept off zero and infinity, and V's type followed what
// all rows see.) More warps only share this out (us, when the first was 53): 16
// softmax warps of 64 keys each 56, 16 unpacking warps 69, 12 in turn 60.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "cache_line.cuh"

namespace lcb {
namespace {

constexpr int kD = 128;
constexpr int kRows = 128, kKeys = 128;  // of a tile, of a unit
constexpr int kProducts = 16, kRecords = 17, kThreads = 18 * 32;  // warps, threads
constexpr uint32_t kTileBytes = 128 * 128 * 2, kHalfBytes = kTileBytes / 2;
constexpr float kRescaleThreshold = 8.0f, kFarScore = 0x1p23f;  // in base 2
constexpr uint32_t kWhere = 10u << 24;

// K's two tiles are those of two units in 4 bits, of one unit's two parts in 8.
template <int BITS>
struct Raw {  // a stage of records
  static constexpr int kStageKeys = BITS == 4 ? 128 : 64, kSubs = kKeys / kStageKeys, kStages = 3;
  static constexpr int kBytes = kStageKeys * cache_row_bytes(BITS);
};

struct Bars {
  uint64_t raw_full[3], raw_empty[3];
  uint64_t q_full;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

template <int BITS>
struct Smem {  // 1024-byte aligned
  uint8_t K[2][kTileBytes], V[2][kTileBytes], Q[kTileBytes];
  uint8_t raw[Raw<BITS>::kStages][Raw<BITS>::kBytes];
  // by unit modulo 4: the power of two taken from K, for each sixteen keys (infinity: each of them has its own); below
  // zero where their V and P are bf16
  float k_factor[4][8];
  float key_factor[4][kKeys];
  uint2 v_nan[4][8];  // and then, of which scales of V are NaN: bits 2 key + G / 2, G even and odd
  float M[2][kRows], L[2][kRows];
  uint32_t nan[2][kRows];
  Bars bars;
  int lens[kLineSequences];
};

// Instruction descriptor, kind::f16, fp32 sums: fp16 operands (format 0).
constexpr uint32_t idesc_f16(int M, int N, bool transposed_b = false) {
  return (1u << 4) | (transposed_b ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Byte offset of 16-byte chunk c (of 8 channels, 16 a row) of row r in a tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * kHalfBytes + static_cast<uint32_t>(r) * 128u +
         (static_cast<uint32_t>((c ^ r) & 7) << 4);
}

__device__ __forceinline__ void st_shared16(uint8_t* at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  *reinterpret_cast<uint4*>(at) = make_uint4(a, b, c, d);
}

__device__ __forceinline__ void fence_to_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

constexpr int kVDown = 12;      // V's tiles hold V times 2^-12,
constexpr float kWeightUp = 7;  // the weights are times 2^7: 2^15 at most, as a maximum may lag by kRescaleThreshold

// A lane (key, t) of eight keys takes its key's channels 32 G + 8 t .. + 7 of all four groups. Eight neighbouring lanes
// have keys four apart: their records' quarters, 144 or 272 bytes a key, and their chunks of the tile's rows lie in
// different banks.
struct Lane {
  int key, t;
  __device__ __forceinline__ explicit Lane(int lane) : key((lane >> 3) | (lane & 4)), t(lane & 3) {}
  // of the first group's chunk in a tile, for rows 8 keys apart
  __device__ __forceinline__ uint32_t first_chunk(int row0) const { return chunk_at(row0 + key, t); }
};
__device__ __forceinline__ uint8_t* chunk_of(uint8_t* tile, uint32_t first, int round, int G) {
  return tile + ((first ^ (G & 1 ? 64u : 0u)) + round * 1024 + (G >> 1) * kHalfBytes);
}

// Whether V of sixteen keys is bf16: `cut`, or a scale is not one for fp16. If so, which scales are NaN (v_nan; an
// infinity, which kv_cache_write never leaves, counts as one).
template <int BITS>
__device__ __forceinline__ bool wide_v(const uint8_t* rec, bool cut, uint2* nan, int lane) {
  const uint32_t x = *reinterpret_cast<const uint32_t*>(rec + (lane >> 1) * cache_row_bytes(BITS) +
                                                        cache_scale_offset(BITS) + 8 + 4 * (lane & 1));
  constexpr uint32_t kLow = (BITS == 4 ? 120u : 116u) << 7, kHigh = 131u << 7;  // 2^-7 or 2^-11, 2^4
  auto out = [](uint32_t a) { return a != 0 && (a < kLow || a >= kHigh); };
  const bool wide = __any_sync(0xffffffffu, cut || out(x & 0xffffu) || out(x >> 16));
  if (wide) {
    const uint32_t even = __ballot_sync(0xffffffffu, (x & 0x7f80u) == 0x7f80u);
    const uint32_t odd = __ballot_sync(0xffffffffu, (x & 0x7f800000u) == 0x7f800000u);
    if (lane == 0) *nan = make_uint2(even, odd);
  }
  return wide;
}

// K's factors are kept times 2^-7, and the rows' times 2^7: 2^(9 + e) passes fp32's end where the largest scales (below
// 2^126, from the largest bf16 over 7) do not, and a row's is 2^119 at most, times the scale.
constexpr int kFactorDown = 7;

// A key's four scales' largest finite one, as bits.
__device__ __forceinline__ uint32_t top_scale(uint32_t x) {
  const uint32_t a = x & 0xffffu, b = x >> 16;
  return max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u);
}

// The exponent of a largest scale given as bits (kv_cache_write leaves none below 2^-107, but zero).
__device__ __forceinline__ int top_exponent(uint32_t top) { return max(static_cast<int>(top >> 7) - 127, -110); }

// Sixteen keys of K by a warp: rows row0 .. + 15 of the tile, times powers of two. OWN: each key its own, which go to
// `own`. Otherwise all of them 2^(-9 - e), e the exponent of their largest scale.
template <int BITS, bool OWN>
__device__ __forceinline__ void unpack_k_rows(const uint8_t* rec, uint8_t* tile, int row0, int e, float* own, int lane) {
  constexpr int kRec = cache_row_bytes(BITS);
  const Lane at(lane);
  const uint8_t* r0 = rec + at.key * kRec;
  const uint32_t first = at.first_chunk(row0);
  // from the codes' 2^-24 (or 2^-20) to 2^-9, with which s goes up to fp16's end
  auto code = [](uint32_t x, bool odd) { return OWN ? hmul2_f16(x, odd ? 0x68006800u : 0x78007800u) : x; };
#pragma unroll(OWN ? 1 : 2)
  for (int round = 0; round < 2; ++round) {
    const uint8_t* r = r0 + round * 8 * kRec;
    const uint2 sc = *reinterpret_cast<const uint2*>(r + cache_scale_offset(BITS));
    if (OWN) {
      e = top_exponent(max(top_scale(sc.x), top_scale(sc.y)));
      if (at.t == 0) own[round * 8 + at.key] = exp2_int(e - 6 - kFactorDown);
    }
    const float up = exp2_int(15 - e);
    uint32_t w[BITS];  // the lane's words
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(r + 64 * i + 16 * at.t);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = j < 2 ? sc.x : sc.y;
      const float f = (j & 1 ? bf16hi_to_f32(x) : bf16lo_to_f32(x)) * up;
      const __half2 d = __floats2half2_rn(f, f);
      const uint32_t s = *reinterpret_cast<const uint32_t*>(&d);
      if (BITS == 4) {
        const uint32_t s16 = OWN ? s : hmul2_f16(s, 0x2c002c00u);  // odd fields are 2^4 as large
        const Fields c = k4_fields(w[j]);
        st_shared16(chunk_of(tile, first, round, j), hmul2_f16(code(c.pair(0), false), s),
                    hmul2_f16(code(c.pair(1), true), s16), hmul2_f16(code(c.pair(2), false), s),
                    hmul2_f16(code(c.pair(3), true), s16));
      } else {
        const uint32_t w0 = w[(2 * j) % BITS], w1 = w[(2 * j + 1) % BITS];
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t keep = part ? 0x800f800fu : 0x80708070u;
          auto value = [&](uint32_t w, int f) { return hmul2_f16(code(k8_f16x2(w, f) & keep, false), s); };
          st_shared16(chunk_of(tile + part * kTileBytes, first, round, j), value(w0, 0), value(w0, 1), value(w1, 0),
                      value(w1, 1));
        }
      }
    }
  }
}

// Sixteen keys of K by a warp; the first nk of the records exist. cut: some row of the tile does not see all sixteen.
template <int BITS>
__device__ __forceinline__ void unpack_k(const uint8_t* rec, uint8_t* tile, int row0, int nk, float* factor, float* own,
                                         uint2* nan, bool cut, int lane, bool& is_wide) {
  constexpr int kRec = cache_row_bytes(BITS);
  uint32_t x = 0;  // half a key's scales
  if ((lane >> 1) < nk)
    x = *reinterpret_cast<const uint32_t*>(rec + (lane >> 1) * kRec + cache_scale_offset(BITS) + 4 * (lane & 1));
  const uint32_t top = __reduce_max_sync(0xffffffffu, top_scale(x));  // the largest finite scale of the sixteen keys
  // the smallest one, less 1 so that zeros are none; whether its exponent is more than 8 below
  const uint32_t low = __reduce_min_sync(0xffffffffu, min((x - 1u) & 0xffffu, ((x >> 16) - 1u) & 0xffffu));
  const bool each = ((low + 1u) >> 7) + 8u < top >> 7;
  const bool wide = wide_v<BITS>(rec, cut, nan, lane);
  is_wide = wide;
  // scales are below 2^(e + 1): times 2^(15 - e) they are fp16, and with the codes' 2^-24 they make s n 2^(-9 - e)
  const int e = top_exponent(top);
  if (lane == 0) *factor = (each ? INFINITY : exp2_int(min(9 - kFactorDown + e, 127))) * (wide ? -1.f : 1.f);
  if (each)
    unpack_k_rows<BITS, true>(rec, tile, row0, 0, own, lane);
  else
    unpack_k_rows<BITS, false>(rec, tile, row0, e, nullptr, lane);
}

// 2^-12 s n of a pair of V's codes, as they lie (magnitudes sh bits to the left). fp16: by one multiplication, by 2^12 s
// over that shift. bf16, for any scale: from the magnitude's 128 + m, by 2^-12 s.
template <bool WIDE>
__device__ __forceinline__ uint32_t v_value(uint32_t code, uint32_t s, int sh) {
  if (!WIDE) return hmul2_f16(code, s);
  const uint32_t m = ((code & 0x7fff7fffu) >> sh) | 0x43004300u;
  return hfma2_bf16(m, s, hmul2_bf16(s, 0xc300c300u)) | (code & 0x80008000u);  // (128 + m) s - 128 s
}
template <bool WIDE>
__device__ __forceinline__ uint32_t v_scales(uint32_t s) {
  if (WIDE) {
    // a NaN's values are zeros here; the rows that see them get theirs at the end (v_nan)
    if ((s & 0x7f80u) == 0x7f80u) s &= 0xffff0000u;
    if ((s & 0x7f800000u) == 0x7f800000u) s &= 0xffffu;
    return hmul2_bf16(s, 0x39803980u);
  }
  const __half2 h = __floats2half2_rn(bf16lo_to_f32(s) * 4096.f, bf16hi_to_f32(s) * 4096.f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Sixteen keys of V, by a warp; keys past the last (of wide ones) become zeros.
template <int BITS, bool WIDE>
__device__ __forceinline__ void unpack_v(const uint8_t* rec, uint8_t* tile, int row0, int nk, int lane) {
  constexpr int kRec = cache_row_bytes(BITS);
  const Lane at(lane);
  const uint8_t* r0 = rec + at.key * kRec;
  const uint32_t first = at.first_chunk(row0);
  constexpr uint32_t kSel[2] = {0x5410, 0x7632};  // of pairs of groups: the first, the second
#pragma unroll
  for (int round = 0; round < 2; ++round) {
    const uint8_t* r = r0 + round * 8 * kRec;
    const uint32_t keep = !WIDE || 8 * round + at.key < nk ? ~0u : 0u;
    const uint2 sc = *reinterpret_cast<const uint2*>(r + cache_scale_offset(BITS) + 8);
    if (BITS == 4) {
      // half-words of lanes 2 t and 2 t + 1: words with groups 0, 1 and 2, 3 of each
      const uint4 v = *reinterpret_cast<const uint4*>(r + cache_v_offset(BITS) + 16 * at.t);
#pragma unroll
      for (int gp = 0; gp < 2; ++gp) {
        const uint32_t s = v_scales<WIDE>(gp ? sc.y : sc.x);
        const uint32_t s16 = WIDE ? s : hmul2_f16(s, 0x2c002c00u);  // odd fields are 2^4 as large
        uint32_t c[2][4];  // channels 4 f + i of both groups
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const Fields x = k4_fields(gp ? (f ? v.w : v.y) : (f ? v.z : v.x));
#pragma unroll
          for (int i = 0; i < 4; ++i) c[f][i] = v_value<WIDE>(x.pair(i), i & 1 ? s16 : s, i & 1 ? 4 : 0);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t sel = kSel[j];
          st_shared16(chunk_of(tile, first, round, 2 * gp + j), permute_bytes(c[0][0], c[0][1], sel) & keep,
                      permute_bytes(c[0][2], c[0][3], sel) & keep, permute_bytes(c[1][0], c[1][1], sel) & keep,
                      permute_bytes(c[1][2], c[1][3], sel) & keep);
        }
      }
    } else {
      const uint32_t s01 = v_scales<WIDE>(sc.x), s23 = v_scales<WIDE>(sc.y);
      uint32_t w[2][4];
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const uint4 v = *reinterpret_cast<const uint4*>(r + cache_v_offset(BITS) + 32 * at.t + 16 * f);
        w[f][0] = v.x, w[f][1] = v.y, w[f][2] = v.z, w[f][3] = v.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t s2 = j < 2 ? s01 : s23;
        const uint32_t s = permute_bytes(s2, s2, j & 1 ? 0x3232 : 0x1010);
        uint32_t o[4];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          o[2 * f] = v_value<WIDE>(permute_bytes(w[f][j], 0, 0x9180) & 0x807f807fu, s, 0) & keep;
          o[2 * f + 1] = v_value<WIDE>(permute_bytes(w[f][j], 0, 0xb3a2) & 0x807f807fu, s, 0) & keep;
        }
        st_shared16(chunk_of(tile, first, round, j), o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// What products of Q and K as they lie in the tiles are times for scores in base 2: a row's factor times a key's. A score
// that the mask hides is -inf before that, which times zero would be NaN, and a score of zero times infinity: neither is
// reached (queries and keys of zeros have the smallest factors that there are).
__device__ __forceinline__ float score_factor(float row, float key) {
  return fminf(fmaxf(row * key, kLeastFactor), 0x1.fffffep127f);
}

// The largest score of a row in a unit, its scores at tS. OWN: some of the keys have powers of two of their own. Without
// it, that is seen from top_factor.
template <bool OWN, class Hidden>
__device__ __forceinline__ float largest(uint32_t tS, const float* k_factor, const float* key_factor, float c, bool whole,
                                         Hidden&& hidden, float& top_factor) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int ch = 0; ch < 4; ++ch) {
    uint32_t s[32];
    tmem_ld_x32(tS + ch * 32, s);
    const float2 kf = *reinterpret_cast<const float2*>(&k_factor[2 * ch]);
    if (!whole)
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (hidden(32 * ch + k)) s[k] = __float_as_uint(-INFINITY);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f16 = fabsf(h ? kf.y : kf.x);
      if (!OWN) top_factor = fmaxf(top_factor, f16);
      if (OWN && f16 == INFINITY) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          mx = fmaxf(mx, __fmul_rn(__uint_as_float(s[16 * h + k]), score_factor(c, key_factor[32 * ch + 16 * h + k])));
        continue;
      }
      float y = -INFINITY, z = -INFINITY;
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        y = fmax3(y, __uint_as_float(s[16 * h + k]), __uint_as_float(s[16 * h + k + 1]));
        z = fmax3(z, __uint_as_float(s[16 * h + k + 2]), __uint_as_float(s[16 * h + k + 3]));
      }
      mx = fmaxf(mx, fmaxf(y, z) * score_factor(c, f16));
    }
  }
  return mx;
}

template <int BITS>
__global__ void __launch_bounds__(kThreads, 1) cache_tiles_kernel(const __grid_constant__ CacheDecode p) {
  using R = Raw<BITS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  auto& sm = *reinterpret_cast<Smem<BITS>*>(smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u));
  Bars& bars = sm.bars;
  volatile int* abort_flag = &bars.abort;
  const int warp = static_cast<int>(uniform(warp_id())), lane = static_cast<int>(lane_id());
  const int cta = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < R::kStages; ++i) {
      mbar_init(&bars.raw_full[i], 1);
      mbar_init(&bars.raw_empty[i], R::kStageKeys / 16);
    }
    mbar_init(&bars.q_full, 8);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars.k_full[t], 8);
      mbar_init(&bars.v_full[t], 8);
      mbar_init(&bars.k_empty[t], 1);
      mbar_init(&bars.v_empty[t], 1);
      mbar_init(&bars.s_full[t], 1);
      mbar_init(&bars.p_full[t], 4);
      mbar_init(&bars.o_full[t], 1);
    }
    mbar_init(&bars.mma_done, 1);
    bars.abort = 0;
    fence_mbar_init();
  }
  copy_lengths(p, sm.lens);
  if (warp == kProducts) {
    tmem_alloc(&bars.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars.tmem_base;
  Walk<kRows, kKeys> walk;
  const bool any = walk.start(p, sm.lens, cta, static_cast<int>(gridDim.x), lane);
  const Tile& a = walk.a;
  // A role's loops: over its tiles, and the units of each. Unit i of the CTA (all tiles together) is stream i % 2's.
  if (any && warp == kRecords) {
    // ------------------------------------------------------------ records
    if (lane == 0) {
      int at = 0;  // stages filled so far
      bool ok = true;
      while (ok && walk.left > 0) {
        const int n = walk.here();
        const uint8_t* head = p.cache + a.b * p.c_bs + a.hk * p.c_hs;
        for (int u = walk.off; u < walk.off + n && ok; ++u) {
          const int j0 = first_key(a, u, kKeys), nk = keys_of(a, u, j0, kKeys);
          for (int s = 0; s < R::kSubs && s * R::kStageKeys < nk; ++s, ++at) {
            const int st = at % R::kStages;
            if (!mbar_wait_inline(&bars.raw_empty[st], (static_cast<uint32_t>(at / R::kStages) & 1u) ^ 1u, abort_flag, p.st,
                                  kWhere | (1u << 16))) {
              ok = false;
              break;
            }
            const uint32_t bytes = static_cast<uint32_t>(min(R::kStageKeys, nk - s * R::kStageKeys)) * cache_row_bytes(BITS);
            mbar_arrive_expect_tx(&bars.raw_full[st], bytes);
            bulk_load(sm.raw[st], head + static_cast<long long>(j0 + s * R::kStageKeys) * cache_row_bytes(BITS), bytes,
                      &bars.raw_full[st]);
          }
        }
        walk.advance(p, sm.lens, n);
      }
      if (!ok)  // copies in flight land before the CTA can end
        for (int k = max(0, at - R::kStages); k < at; ++k)
          drain_wait(&bars.raw_full[k % R::kStages], static_cast<uint32_t>(k / R::kStages) & 1u, p.st.limit);
    }
    __syncwarp();
  } else if (any && warp >= 8 && warp < kProducts) {
    // ------------------------------------------------------------ unpack
    const int w = warp - 8, row0 = 16 * w;
    int stage = 0;  // of the unit's first records
    bool ok = true;
    for (int i = 0; ok && walk.left > 0;) {
      const int n = walk.here();
      for (int u = walk.off; u < walk.off + n && ok; ++u, ++i) {
        const int j0 = first_key(a, u, kKeys), nk = keys_of(a, u, j0, kKeys);
        const int t = i & 1, kt = BITS == 4 ? t : 0;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1u;
        const int sub = row0 / R::kStageKeys, mine = nk - row0;  // the warp's keys that exist, of 16
        const int st = (stage + sub) % R::kStages;
        const uint8_t* rec = sm.raw[st] + (row0 % R::kStageKeys) * cache_row_bytes(BITS);
        const bool loaded = sub * R::kStageKeys < nk;
        if (loaded)
          ok = mbar_wait_warp(&bars.raw_full[st], static_cast<uint32_t>((stage + sub) / R::kStages) & 1u, abort_flag, p.st,
                              kWhere | (2u << 16));
        if (ok)
          ok = mbar_wait_warp(&bars.k_empty[kt], (BITS == 4 ? ph : static_cast<uint32_t>(i) & 1u) ^ 1u, abort_flag, p.st,
                              kWhere | (3u << 16));
        if (!ok) break;
        // whether some row of the tile does not see all sixteen
        const int k0 = j0 + row0, k1 = k0 + 15;
        const bool cut = mine < 16 || k1 > a.p_min || (k0 <= a.p_max - p.window && k1 >= p.sinks);
        bool wide = true;
        if (mine > 0)
          unpack_k<BITS>(rec, sm.K[kt], row0, mine, &sm.k_factor[i & 3][w], &sm.key_factor[i & 3][row0],
                         &sm.v_nan[i & 3][w], cut, lane, wide);
        else if (lane == 0)
          sm.k_factor[i & 3][w] = -1.f, sm.v_nan[i & 3][w] = make_uint2(0, 0);
        fence_to_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.k_full[kt]);
        ok = mbar_wait_warp(&bars.v_empty[t], ph ^ 1u, abort_flag, p.st, kWhere | (4u << 16));
        if (!ok) break;
        if (wide)
          unpack_v<BITS, true>(rec, sm.V[t], row0, mine, lane);
        else
          unpack_v<BITS, false>(rec, sm.V[t], row0, mine, lane);
        fence_to_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.v_full[t]);
          if (loaded) mbar_arrive(&bars.raw_empty[st]);
        }
        stage += (nk + R::kStageKeys - 1) / R::kStageKeys;
      }
      walk.advance(p, sm.lens, n);
    }
  } else if (any && warp == kProducts) {
    // ------------------------------------------------------------ products
    const uint32_t elected = elect_one();
    const uint32_t idesc_qk = idesc_f16(kRows, kKeys), idesc_pv = idesc_f16(kRows, kD, true),
                   idesc_pv_wide = idesc_bf16(kRows, kD, false, true);
    const uint32_t sQ = uniform(smem_u32(sm.Q)), sK = uniform(smem_u32(sm.K)), sV = uniform(smem_u32(sm.V));
    const uint32_t tb = uniform(tbase);
    int seg = 0;
    bool ok = true;
    for (int i0 = 0; ok && walk.left > 0; ++seg) {
      const int n = walk.here();
      ok = mbar_wait_warp(&bars.q_full, static_cast<uint32_t>(seg) & 1u, abort_flag, p.st, kWhere | (5u << 16));
      if (!ok) break;
      tc_fence_after();
      for (int x = 0; x <= n && ok; ++x) {
        if (x < n) {  // S of unit x; the weights of unit x - 2, in its place, have been issued
          const int i = i0 + x, t = i & 1;
          const int kt = BITS == 4 ? t : 0;
          ok = mbar_wait_warp(&bars.k_full[kt], static_cast<uint32_t>(BITS == 4 ? i >> 1 : i) & 1u, abort_flag, p.st,
                              kWhere | (6u << 16));
          if (!ok) break;
          tc_fence_after();
          const uint64_t qa = sdesc_sw128(sQ, 16, 1024);
#pragma unroll
          for (int part = 0; part < BITS / 4; ++part) {
            const uint64_t kb = sdesc_sw128(sK + (kt + part) * kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
              const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
              mma_ss_if(tb + t * 128, sdesc_advance(qa, off), sdesc_advance(kb, off), idesc_qk, part + kk > 0, elected);
            }
          }
          tc_commit_if(&bars.s_full[t], elected);
          tc_commit_if(&bars.k_empty[kt], elected);
        }
        if (x > 0) {  // O of unit x - 1
          const int i = i0 + x - 1, t = i & 1;
          const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1u;
          ok = mbar_wait_warp(&bars.v_full[t], ph, abort_flag, p.st, kWhere | (7u << 16)) &&
               mbar_wait_warp(&bars.p_full[t], ph, abort_flag, p.st, kWhere | (8u << 16));
          if (!ok) break;
          tc_fence_after();
          const uint64_t vb = sdesc_sw128(sV + t * kTileBytes, kHalfBytes, 1024);
          const uint32_t wide = __ballot_sync(0xffffffffu, lane < 8 && sm.k_factor[i & 3][lane & 7] < 0.f);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_ts_if(tb + 256 + t * 128, tb + t * 128 + kk * 8, sdesc_advance(vb, kk * 2048),
                      wide >> kk & 1u ? idesc_pv_wide : idesc_pv, x > 2 || kk > 0, elected);
          tc_commit_if(&bars.v_empty[t], elected);
          if (x + 2 > n) tc_commit_if(&bars.o_full[t], elected);  // the stream's last in this tile
        }
      }
      i0 += n;
      walk.advance(p, sm.lens, n);
    }
    // every product issued must finish before tensor memory is released
    tc_commit_if(&bars.mma_done, elected);
    drain_wait(&bars.mma_done, 0, p.st.limit);
    __syncwarp();
  } else if (any && warp < 8) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + t * 128 + lane_off, tO = tbase + 256 + lane_off;
    uint32_t o_phase = 0;
    bool ok = true;
    float* slot = p.workspace + 2LL * cta * slot_floats(kRows);
    for (int i0 = 0, seg = 0; walk.left > 0; ++seg) {
      const int n = walk.here();
      const int R_all = p.T * p.G, r = a.r0 + row;
      const bool active = a.r0 + (warp & 3) * 32 < R_all;  // the warp has a row
      const int tok = r / p.G;
      const int pos = r < R_all ? a.p0 + tok : -1;
      // ---- Q: this stream's half of the channels, over the power of two of the whole row
      float c;
      {
        const __nv_bfloat16* src =
            p.q + a.b * p.q_bs + static_cast<long long>(tok) * p.q_rs + (a.hk * p.G + r - tok * p.G) * kD;
        uint32_t top = 0;
        if (r < R_all)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * k);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(x[j] & 0x7fffu, x[j] >> 16 & 0x7fffu));
          }
        const int e = static_cast<int>(top >> 7), up = min(126, kQTop + 127 - e);
        const float f = e == 255 ? __int_as_float(0x7fc00000) : exp2_int(up);
        c = exp2_int(kFactorDown - up) * p.scale_log2;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (r < R_all) v = *reinterpret_cast<const uint4*>(src + 64 * t + 8 * k);
          const uint32_t x[4] = {v.x, v.y, v.z, v.w};
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 h = __floats2half2_rn(bf16lo_to_f32(x[j]) * f, bf16hi_to_f32(x[j]) * f);
            y[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          st_shared16(sm.Q + chunk_at(row, 8 * t + k), y[0], y[1], y[2], y[3]);
        }
      }
      fence_to_async();
      tc_fence_before();  // and the last tile's sums have been read
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full);
      float m = -INFINITY, l = 0.f;
      bool any_far = false;
      uint32_t row_nan = 0;  // channel groups in which the row sees a NaN of V
      auto spread = [](uint32_t two) { return (two & 1u) | (two & 2u) << 1; };  // groups 0, 2
      const int first = (i0 & 1) == t ? 0 : 1;  // the stream's first unit of the tile
      for (int x = first; x < n && ok; x += 2) {
        const int i = i0 + x;
        const uint32_t ph = static_cast<uint32_t>(i >> 1) & 1u;
        // (k_factor too: it was stored before the arrivals that these products waited for)
        ok = mbar_wait_warp(&bars.s_full[t], ph, abort_flag, p.st, kWhere | (9u << 16));
        if (!ok) break;
        tc_fence_after();
        if (active) {
          const int u = walk.off + x;
          const bool whole = u >= a.whole0 && u < a.whole1;
          const int j0 = first_key(a, u, kKeys), nk = keys_of(a, u, j0, kKeys);
          auto hidden = [&](int k) {
            const int j = j0 + k;
            return !(k < nk && j <= pos && (pos - j < p.window || j < p.sinks));
          };
          // Some of the keys may have powers of two of their own: copies of the loops, which few units take. (64 rows x 64K
          // keys, us: without such keys 46.9; with a test in the loops 52.2; so 48.8.)
          float top_factor = 0.f;
          float mx = largest<false>(tS, sm.k_factor[i & 3], sm.key_factor[i & 3], c, whole, hidden, top_factor);
          const bool own = top_factor == INFINITY;
          if (own) mx = largest<true>(tS, sm.k_factor[i & 3], sm.key_factor[i & 3], c, whole, hidden, top_factor);
          const float m_new = fmaxf(m, mx);
          const bool resc = m_new > m + kRescaleThreshold;
          // A row whose maximum is so large that the rounding of the product it was is no longer small beside 1: its
          // weights take a multiplication and a subtraction. Whether the warp has one changes with the maxima alone.
          auto is_far = [&] { return fabsf(m) >= kFarScore && m != -INFINITY; };
          if (x == first) {
            m = m_new;
            any_far = __any_sync(0xffffffffu, is_far());
          } else if (__any_sync(0xffffffffu, resc)) {
            const float alpha = resc ? ex2_approx(m - m_new) : 1.f;
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t o[32];
              tmem_ld_x32(tO + t * 128 + ch * 32, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st_x32(tO + t * 128 + ch * 32, o);
            }
            if (resc) {
              l *= alpha;
              m = m_new;
            }
            any_far = __any_sync(0xffffffffu, is_far());
          }
          const float neg_m = m == -INFINITY ? 0.f : kWeightUp - m;
          auto weights = [&](auto rare) {
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t s[32], pk[16];
              tmem_ld_x32(tS + ch * 32, s);
              const float2 kf = *reinterpret_cast<const float2*>(&sm.k_factor[i & 3][2 * ch]);
              if (!whole)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (hidden(32 * ch + k)) s[k] = __float_as_uint(-INFINITY);
              float la = 0.f, lb = 0.f;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float f16 = fabsf(h ? kf.y : kf.x), f = score_factor(c, f16);
                const float* own = &sm.key_factor[i & 3][32 * ch + 16 * h];
                float w[16];
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                  const float s0 = __uint_as_float(s[16 * h + k]), s1 = __uint_as_float(s[16 * h + k + 1]);
                  float f0 = f, f1 = f;
                  if (rare.value && f16 == INFINITY) f0 = score_factor(c, own[k]), f1 = score_factor(c, own[k + 1]);
                  ffma2(w[k], w[k + 1], s0, s1, f0, f1, neg_m, neg_m);
                  if (rare.value && is_far()) {
                    w[k] = __fsub_rn(__fmul_rn(s0, f0), m) + kWeightUp;
                    w[k + 1] = __fsub_rn(__fmul_rn(s1, f1), m) + kWeightUp;
                  }
                  w[k] = ex2_approx(w[k]), w[k + 1] = ex2_approx(w[k + 1]);
                  fadd2(la, lb, la, lb, w[k], w[k + 1]);
                }
                if ((h ? kf.y : kf.x) < 0.f) {
                  const uint2 nan = sm.v_nan[i & 3][2 * ch + h];
                  if ((nan.x | nan.y) != 0)  // V's NaN, as far as the row sees their keys
#pragma unroll 1
                    for (int k = 0; k < 16; ++k)
                      if (!hidden(32 * ch + 16 * h + k))
                        row_nan |= spread(nan.x >> 2 * k) | spread(nan.y >> 2 * k) << 1;
#pragma unroll
                  for (int k = 0; k < 8; ++k) pk[8 * h + k] = pack_bf16x2(w[2 * k], w[2 * k + 1]);
                } else {
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const __half2 x = __floats2half2_rn(w[2 * k], w[2 * k + 1]);
                    pk[8 * h + k] = *reinterpret_cast<const uint32_t*>(&x);
                  }
                }
              }
              l += la + lb;
              tmem_st_x16(tS + ch * 16, pk);  // over scores that have been read
            }
          };
          if (own || any_far)
            weights(std::true_type());
          else
            weights(std::false_type());
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t]);
      }
      if (ok && first < n) {
        ok = mbar_wait_warp(&bars.o_full[t], o_phase, abort_flag, p.st, kWhere | (10u << 16));
        o_phase ^= 1u;
      }
      m -= kWeightUp;  // what the weights and sums are relative to
      sm.M[t][row] = m;
      sm.L[t][row] = l;
      sm.nan[t][row] = row_nan;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      tc_fence_after();
      // ---- both streams' parts of the row, channels 64 t .. + 63
      const float m2 = sm.M[1 - t][row], l2 = sm.L[1 - t][row];
      const float M = fmaxf(m, m2), f = weight(m, M), f2 = weight(m2, M), L = t == 0 ? f * l + f2 * l2 : f2 * l2 + f * l;
      const bool whole_tile = n == a.units, have = first < n, have2 = n > 1 || !have;
      if (active && ok) {
        const float inv = exp2_int(kVDown) * (!whole_tile ? 1.f : L == 0.f ? 0.f : 1.f / L);
        const float g0 = (t == 0 ? f : f2) * inv, g1 = (t == 0 ? f2 : f) * inv;
        // a stream without units in this tile, or without a key that the row sees, has nothing to add
        const bool mine = have && l != 0.f, other = have2 && l2 != 0.f;
        const bool have_0 = t == 0 ? mine : other, have_1 = t == 0 ? other : mine;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t x[16], y[16];
          tmem_ld_x16(tO + 64 * t + 16 * ch, x);
          tmem_ld_x16(tO + 128 + 64 * t + 16 * ch, y);
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = (have_0 ? g0 * __uint_as_float(x[k]) : 0.f) + (have_1 ? g1 * __uint_as_float(y[k]) : 0.f);
          if ((sm.nan[0][row] | sm.nan[1][row]) >> (2 * t + (ch >> 1)) & 1u)
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __int_as_float(0x7fc00000);
          if (r < R_all) {
            if (whole_tile) {
              __nv_bfloat16* dst = p.o + a.b * p.o_bs + static_cast<long long>(tok) * p.o_rs +
                                   (a.hk * p.G + r - tok * p.G) * kD + 64 * t + 16 * ch;
#pragma unroll
              for (int k = 0; k < 16; k += 8)
                *reinterpret_cast<uint4*>(dst + k) =
                    make_uint4(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]),
                               pack_bf16x2(v[k + 4], v[k + 5]), pack_bf16x2(v[k + 6], v[k + 7]));
            } else {
              float* dst = slot + row * kD + 64 * t + 16 * ch;
#pragma unroll
              for (int k = 0; k < 16; k += 4)
                *reinterpret_cast<float4*>(dst + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
          }
        }
        if (t == 0 && r < R_all) {
          if (whole_tile) {
            p.lse[a.b * p.l_bs + (a.hk * p.G + r - tok * p.G) * p.l_hs + tok] =
                L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
          } else {
            slot[kRows * kD + row] = M;
            slot[kRows * (kD + 1) + row] = L;
          }
        }
      }
      i0 += n;
      walk.advance(p, sm.lens, n);
      slot = p.workspace + (2LL * cta + 1) * slot_floats(kRows);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // M, L and the sums have been read, Q's products are done
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProducts) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int BITS>
struct TilesForm {
  static constexpr int kSmem = sizeof(Smem<BITS>) + 1024;
  static const void* fn() { return reinterpret_cast<const void*>(cache_tiles_kernel<BITS>); }

  static DeviceOnce& allowed() {
    static DeviceOnce once;
    return once;
  }

  static int ctas(const ContextKey& at) {
    static ClusterCounts known;
    return resident_clusters(known, at, allowed(), fn(), kThreads, kSmem, 1);
  }
};

}  // namespace

int cache_tiles_ctas(int bits, const ContextKey& at) {
  return bits == 4 ? TilesForm<4>::ctas(at) : TilesForm<8>::ctas(at);
}

size_t cache_tiles_workspace(int ctas) { return 2 * sizeof(float) * slot_floats(kRows) * static_cast<size_t>(ctas); }

template <int BITS>
static int launch(const CacheDecode& p, long long tiles, int ctas, cudaStream_t stream) {
  const int rc = set_smem_limit_once(TilesForm<BITS>::allowed(), TilesForm<BITS>::fn(), TilesForm<BITS>::kSmem);
  if (rc != 0) return rc;
  cache_tiles_kernel<BITS><<<ctas, kThreads, TilesForm<BITS>::kSmem, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return -4;
  return launch_cache_join<kRows, kKeys>(p, tiles, ctas, stream);
}

int launch_cache_tiles(CacheDecode p, int bits, int ctas, cudaStream_t stream) {
  p.G = p.H / p.Hkv;
  p.row_tiles = static_cast<int>((static_cast<long long>(p.T) * p.G + kRows - 1) / kRows);
  p.cluster = 1;
  const long long tiles = static_cast<long long>(p.B) * p.Hkv * p.row_tiles;
  return bits == 4 ? launch<4>(p, tiles, ctas, stream) : launch<8>(p, tiles, ctas, stream);
}

}  // namespace lcb
