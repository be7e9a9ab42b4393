// Attention of the newest tokens over a quantised K/V cache (kv_cache.cuh),
// with the mask of the windowed attention: the query at position p sees keys
// j <= p with p - j < window, and the first `sinks` keys.
//
// A cached row holds, per group G of 32 channels, whole numbers and a scale:
//   k_jc = s^K_jG n_jc,   x_ij = scale * sum_G s^K_jG sum_{c in G} q_ic n_jc
//   v_jc = s^V_jG n_jc,   o_ic = sum_j (p_ij s^V_jG) n_jc / l_i
// so the products take the whole numbers, which 8 or 16 bits hold exactly, and
// the scales go to the scores and to the weights: nothing of the cache is
// rounded. p s^V goes to bf16 for the second product, as P does in the other
// forms: half a step, up to 2^-8 of each weight, of either sign. Q goes to fp16
// for the first one, after a division by a power of two that puts a row's
// largest element into [2^15, 2^16), or [2^11, 2^12) in the half of the channels whose
// 4-bit codes lie 2^4 higher: exact but for elements below 2^-28 of that largest, whose
// errors are under 2^-36 of it.
//
// Every visible record (144 or 272 bytes) is read once for all query rows that
// share its head, up to 16 of them. HBM bounds it only if little is done per
// byte: at 6.7 TB/s an SM gets a 4-bit key every 6 clocks, 24 issue slots for
// its 256 numbers. Hence
//   S^T[16 keys][8 rows] = K Q^T  and  O^T[128][8 rows] += V^T P^T  on warp
//     mma.sync (m16n8k16) with operands in registers, as attn_window_split.cu.
//     tcgen05 would want its operand unpacked into shared or tensor memory, and
//     8-bit products (m16n8k32) are two 16-bit ones and conversions here;
//   codes stored as parts of subnormal numbers in operand order, so that little
//     more than an AND makes a register of them an operand (kv_cache.cuh). The
//     smallness is made up for by Q's power of two and the scores' factor, and
//     for V by weights times 2^96 (less while scales are so large that those
//     would not fit), taken back when the parts are joined;
//   records brought to shared memory by bulk copies, one instruction for
//     several KB: no address arithmetic.
//
// Two forms share that loop. With few keys in all, a cluster of CTAs takes a
// (sequence, K/V head, row tile), its keys dealt evenly to the cluster's warps,
// whose partial (m, l, O) are joined in shared memory, then through distributed
// shared memory: one launch, no workspace. With more, the units of all tiles
// form one line that is cut into equal pieces, one for each CTA that the GPU
// holds, whatever the lengths and however few the heads; a CTA walks over its
// piece tile by tile, and pieces of a tile that several CTAs share go to a
// workspace, which a second kernel joins. No atomics: the same result every
// time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "cache_line.cuh"
#include "lcb_attn.h"

namespace cg = cooperative_groups;

namespace lcb {
namespace {

constexpr int kD = 128;
constexpr int kStep = 16;  // keys of a product, and of a warp's turn
constexpr float kRescaleThreshold = 8.0f;  // log2 units: the running maximum is raised lazily, P stays <= 256
constexpr uint32_t kWhere = 9u << 24;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// mma_f16 with nothing to add to.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// How a tile of ROWS query rows lies in the eight columns of a product, and
// what a lane (g, t) has of them.
//   8, 16: a column is a row; lane t has the rows 2t and 2t + 1 of every eight.
//     The scores come as four sums, one for each group of channels, and a
//     weight goes into the second product four times, once with each scale.
//   4: a column 2r + h is half h of row r: the groups 2h and 2h + 1, Q being zero
//     in the other half. So two sums and two operands do where eight columns of
//     whole rows take four, and lane t has row t alone: 260 instructions for
//     sixteen keys in 4 bits in the line form (eight rows: 325).
template <int ROWS>
struct Cols {
  static constexpr bool kHalves = ROWS == 4;
  static constexpr int kTiles = ROWS == 16 ? 2 : 1;          // eights of columns
  static constexpr int kMine = kHalves ? 1 : 2 * kTiles;     // rows of a lane
  static constexpr int kSums = kHalves ? 2 : 4;              // sums, and operands, per eight columns
  static __device__ int row(int i, int t) { return kHalves ? t : 8 * (i >> 1) + 2 * t + (i & 1); }  // a lane's i-th
};

constexpr int kUp = 96;            // weights go into the second product times 2^96, which subnormal codes take back
constexpr int kUpRange = 119 - kUp;  // while V's scales are below 2^23: a weight is 2^8 at most

// A row is far where one fused multiplication does not make weights of its products: where its factor could pass fp32's
// end (a largest |q| of 2^76 or more), or where its maximum is so large that the rounding of the product it was is no
// longer small beside 1. Its raise_at stays -inf, so that every step takes the branch that raises a maximum, and there
// its products become differences from m, by a multiplication and a subtraction, over c. Such a row's c is its factor
// over 2^24, and its neg_m -0, which no other row's is. (With the factor in a register of its own: 8 heads x 65536
// keys, sixteen rows, 8 bits 50.4 us for 49.6; 46.8 without far rows.)
constexpr float kFarScore = 0x1p23f;
__device__ __forceinline__ bool is_far(float neg_m) { return __float_as_uint(neg_m) == 0x80000000u; }

template <int ROWS, int BITS>
struct State {
  using C = Cols<ROWS>;
  uint32_t q[C::kTiles][16];    // Q's fragments, in K's channel order
  float c[C::kMine];            // a row's scores in base 2 are its products times this (a far row's 2^24 more)
  int pr[C::kMine];             // its position; -1 past the last row
  float o[8][C::kTiles][4];     // o[2 G + f]: channels 32 G + 4 g + 2 f + {0, 1}, each of columns 2t, 2t + 1
  float m[C::kMine], l[C::kMine];
  float neg_m[C::kMine], raise_at[C::kMine];  // -m (0 while nothing is seen); the product above which m is raised
  float up[C::kMine];           // what a row's weights go into the second product with: 2^kUp, or less
  uint32_t up_limit;            // bf16, twice: V's scales above it want a smaller one, of some row that sees them
  // O of a lane's row i in channel 32 G + 4 g + k, times `up` and a subnormal's factor
  __device__ float& out(int i, int G, int k) {
    const int col = C::kHalves ? G >> 1 : i & 1;
    return o[2 * G + (k >> 1)][C::kHalves ? 0 : i >> 1][2 * (k & 1) + col];
  }
  __device__ float true_out(int i, int G, int k, float down) {
    return out(i, G, k) * (BITS == 4 && (k & 1) ? 0x1p61f : 0x1p65f) * down;
  }
  __device__ int up_exponent(int i) const { return static_cast<int>(__float_as_uint(up[i]) >> 23) - 127; }
  // 2^68 / up: an exponent of at most 85
  __device__ float down(int i) const { return exp2_int(68 - up_exponent(i)); }
};

// A lane's part of Q as it lies in memory.
template <int ROWS>
struct RawQ {
  uint4 v[Cols<ROWS>::kTiles][Cols<ROWS>::kHalves ? 2 : 4];
};

template <int ROWS>
__device__ __forceinline__ RawQ<ROWS> load_q(const CacheDecode& p, const Tile& a, int g, int t) {
  using C = Cols<ROWS>;
  RawQ<ROWS> x;
#pragma unroll
  for (int nt = 0; nt < C::kTiles; ++nt) {
    const int r = a.r0 + (C::kHalves ? g >> 1 : 8 * nt + g);
    const int tok = p.G == 1 ? r : r / p.G;
    const __nv_bfloat16* src = p.q + a.b * p.q_bs + static_cast<long long>(tok) * p.q_rs +
                               (a.hk * p.G + r - tok * p.G) * kD + 8 * t + (C::kHalves ? 64 * (g & 1) : 0);
#pragma unroll
    for (int c = 0; c < (C::kHalves ? 2 : 4); ++c)
      x.v[nt][c] = r < p.T * p.G ? *reinterpret_cast<const uint4*>(src + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
  }
  return x;
}

template <int ROWS, int BITS>
__device__ __forceinline__ void begin(State<ROWS, BITS>& w, const RawQ<ROWS>& raw, const CacheDecode& p, const Tile& a,
                                      int g, int t) {
  using C = Cols<ROWS>;
  constexpr int kLoaded = C::kHalves ? 2 : 4;  // groups that the lane has
#pragma unroll
  for (int nt = 0; nt < C::kTiles; ++nt) {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < kLoaded; ++c) {
      const uint32_t x[4] = {raw.v[nt][c].x, raw.v[nt][c].y, raw.v[nt][c].z, raw.v[nt][c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7fffu, x[i] >> 16 & 0x7fffu));
    }
#pragma unroll
    for (int x = 1; x < (C::kHalves ? 8 : 4); x *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
    const int e = static_cast<int>(top >> 7);  // 127 more than the exponent; 255 with infinities or NaN
    const int up = min(126, kQTop + 127 - e);
    const float f = e == 255 ? __int_as_float(0x7fc00000) : exp2_int(up);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = raw.v[nt][C::kHalves ? c & 1 : c];
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      const bool zero = C::kHalves && (c >> 1) != (g & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float fi = BITS == 4 && (i & 1) ? f * 0.0625f : f;  // those codes are 2^4 as large
        const __half2 y = __floats2half2_rn(bf16lo_to_f32(x[i]) * fi, bf16hi_to_f32(x[i]) * fi);
        w.q[nt][4 * c + i] = zero ? 0u : *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    // the power of two back, and the subnormal codes' 2^24
    auto factor = [&](int i, int up) {
      const float all = exp2_int(min(24 - up, 127)) * p.scale_log2;
      const bool far = up < -60 || all >= 0x1p84f;
      // (zero times a hidden score's -inf would be NaN)
      w.c[i] = far ? fminf(exp2_int(-up) * p.scale_log2, 0x1p125f) : fmaxf(all, kLeastFactor);
      w.neg_m[i] = far ? -0.f : 0.f;
    };
    if (C::kHalves) {
      factor(0, __shfl_sync(0xffffffffu, up, 8 * t));
    } else {
      factor(2 * nt, __shfl_sync(0xffffffffu, up, 8 * t));
      factor(C::kMine > 1 ? 2 * nt + 1 : 0, __shfl_sync(0xffffffffu, up, 8 * t + 4));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) w.o[i][nt][k] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < C::kMine; ++i) {
    const int r = a.r0 + C::row(i, t);
    w.pr[i] = r < p.T * p.G ? a.p0 + (p.G == 1 ? r : r / p.G) : -1;
    w.m[i] = w.raise_at[i] = -INFINITY;
    w.l[i] = 0.f;
    w.up[i] = exp2_int(kUp);
  }
  w.up_limit = 0x10001u * ((kUpRange + 127) * 128 - 1);
}

// The largest scale of V, as bits, for which a weight times 2^(119 - range) times it is a number: below 2^range.
__device__ __forceinline__ uint32_t scale_limit(int range) { return range >= 128 ? 0x7f7fu : (range + 127) * 128 - 1; }

// Some scales of V (of the lane's two keys) are so large that weights times `up` would not fit: for each row, the smaller
// `up` that the largest one that it sees needs. (A key that it does not see takes nothing of its precision.) NaN is none
// of them. `sees` tells whether the lane's row i sees its key h.
template <int ROWS, int BITS, class Sees>
__device__ __forceinline__ void lower_up(State<ROWS, BITS>& w, const uint4 (&sc)[2], Sees&& sees) {
  using C = Cols<ROWS>;
  uint32_t top[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    top[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = i < 2 ? sc[h].z : sc[h].w, s = i & 1 ? x >> 16 : x & 0xffffu;
      top[h] = max(top[h], s < 0x7f80u ? s : 0u);
    }
  }
  if (__reduce_max_sync(0xffffffffu, max(top[0], top[1])) <= (w.up_limit & 0xffffu)) return;
  uint32_t limit = 0xffffu;
#pragma unroll
  for (int i = 0; i < C::kMine; ++i) {
    uint32_t seen = max(sees(0, i) ? top[0] : 0u, sees(1, i) ? top[1] : 0u);
    for (int x = 4; x < 32; x *= 2) seen = max(seen, __shfl_xor_sync(0xffffffffu, seen, x));
    float f = 1.f;
    if (seen > scale_limit(119 - w.up_exponent(i))) {
      const int e = static_cast<int>(seen >> 7) - 126;      // scales below 2^e
      const float up = exp2_int(119 - min(e + 8, 128));     // room for some growth
      f = up / w.up[i];
      w.up[i] = up;
    }
    limit = min(limit, scale_limit(119 - w.up_exponent(i)));
#pragma unroll
    for (int G = 0; G < 4; ++G)
#pragma unroll
      for (int k = 0; k < 4; ++k) w.out(i, G, k) *= f;
  }
  w.up_limit = 0x10001u * __reduce_min_sync(0xffffffffu, limit);
}

// Which of a step's sixteen keys is row x + 8 h of the first product, and so the second one's x + 8 h along the sum: rows
// 2 m and 2 m + 1 are four keys apart modulo eight, rows 0, 2, 4, 6 two and 1, 3, 5, 7 two. A record is four banks past
// a multiple of 32, so that neither product's loads have two lanes in one bank.
__device__ __forceinline__ int key_of(int x, int h) { return (x & 1 ? 8 + ((x + 3) & 7) : x) + h; }

// Sixteen keys at `rec`, the first nk of which exist: key j0 + i of the
// sequence at i. CUT: some of them may be hidden from some rows.
template <int ROWS, int BITS, bool CUT>
__device__ __forceinline__ void step(State<ROWS, BITS>& w, const CacheDecode& p, const uint8_t* rec, int j0, int nk, int g,
                                     int t) {
  using C = Cols<ROWS>;
  constexpr int kRec = cache_row_bytes(BITS), kWords = BITS / 4;  // of a group, for a lane
  // the lane's keys of the first product, and their scales: four of K, four of V
  const int key0 = key_of(g, 0);
  const uint8_t* mine = rec + key0 * kRec;
  uint4 sc[2] = {*reinterpret_cast<const uint4*>(mine + cache_scale_offset(BITS)),
                 *reinterpret_cast<const uint4*>(mine + kRec + cache_scale_offset(BITS))};
  if (CUT) {
    if (key0 >= nk) sc[0].z = sc[0].w = 0u;
    if (key0 + 1 >= nk) sc[1].z = sc[1].w = 0u;
  }
  auto k_scale = [&](int h, int c) {
    const uint32_t x = c < 2 ? sc[h].x : sc[h].y;
    return c & 1 ? bf16hi_to_f32(x) : bf16lo_to_f32(x);
  };
  auto v_scale = [&](int h, int c) {
    const uint32_t x = c < 2 ? sc[h].z : sc[h].w;
    return c & 1 ? bf16hi_to_f32(x) : bf16lo_to_f32(x);
  };
  // ---- S^T: s[h][i] is key_of(g, h), the lane's row i
  float s[2][C::kMine];
  {
    uint32_t kw[2][4 * kWords];  // a key's words: one, or two, of each group
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(mine + h * kRec + 64 * i + 16 * t);
        kw[h][4 * i] = v.x;
        kw[h][4 * i + 1] = v.y;
        kw[h][4 * i + 2] = v.z;
        kw[h][4 * i + 3] = v.w;
      }
    float acc[C::kSums][C::kTiles][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t x[2][4];  // pairs of channels of the lane's two keys
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Fields f = k4_fields(kw[h][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[h][i] = BITS == 4 ? f.pair(i) : k8_f16x2(kw[h][(2 * c + (i >> 1)) % (4 * kWords)], i & 1);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < C::kTiles; ++nt) {
          const uint32_t b0 = w.q[nt][4 * c + 2 * h], b1 = w.q[nt][4 * c + 2 * h + 1];
          if (h == 0 && c < C::kSums)
            mma_f16_first(acc[c][nt], x[0][2 * h], x[1][2 * h], x[0][2 * h + 1], x[1][2 * h + 1], b0, b1);
          else
            mma_f16(acc[c % C::kSums][nt], x[0][2 * h], x[1][2 * h], x[0][2 * h + 1], x[1][2 * h + 1], b0, b1);
        }
      if (!C::kHalves)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < C::kMine; ++i) {
            const float x = acc[c % C::kSums][i >> 1][2 * h + (i & 1)];
            s[h][i] = c == 0 ? k_scale(h, c) * x : fmaf(k_scale(h, c), x, s[h][i]);
          }
    }
    if (C::kHalves)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        s[h][0] = fmaf(k_scale(h, 3), acc[1][0][2 * h + 1],
                       fmaf(k_scale(h, 2), acc[0][0][2 * h + 1],
                            fmaf(k_scale(h, 1), acc[1][0][2 * h], k_scale(h, 0) * acc[0][0][2 * h])));
  }
  bool seen[2][C::kMine];
  if (CUT) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = key0 + h, j = j0 + i;
#pragma unroll
      for (int x = 0; x < C::kMine; ++x) {
        const int pp = w.pr[x];
        seen[h][x] = i < nk && j <= pp && (pp - j < p.window || j < p.sinks);
        if (!seen[h][x]) s[h][x] = -INFINITY;
      }
    }
  }
  uint32_t vw[4][2 * kWords];  // V's words of rows 2t, 2t + 1, 2t + 8, 2t + 9
  auto load_v = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* at = rec + key_of(2 * t + (i & 1), i >> 1) * kRec + cache_v_offset(BITS) + 2 * BITS * g;
      if (BITS == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        vw[i][0] = v.x;
        vw[i][1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        vw[i][0] = v.x;
        vw[i][1] = v.y;
        vw[i][(2 * kWords) - 2] = v.z;
        vw[i][(2 * kWords) - 1] = v.w;
      }
    }
  };
  // before the branch with eight rows, so that they arrive during the weights (us, so / after: 8 x 2 tokens of 8 x 20001
  // keys 36.2 / 37.6; with four rows 8 heads x 524288 101 / 99)
  if (ROWS == 8) load_v();
  bool raise = false;
#pragma unroll
  for (int i = 0; i < C::kMine; ++i) raise |= s[0][i] > w.raise_at[i] || s[1][i] > w.raise_at[i];
  const uint32_t v_top = max_u16x2(max_u16x2(sc[0].z, sc[0].w), max_u16x2(sc[1].z, sc[1].w));
  raise |= max_u16x2(v_top, w.up_limit) != w.up_limit;
  if (__any_sync(0xffffffffu, raise)) {
    lower_up(w, sc, [&](int h, int i) { return !CUT || seen[h][i]; });
#pragma unroll
    for (int i = 0; i < C::kMine; ++i) {
      const bool was_far = is_far(w.neg_m[i]);
      float mx = fmaxf(s[0][i], s[1][i]) * w.c[i] * (was_far ? 0x1p24f : 1.f);
#pragma unroll
      for (int x = 4; x < 32; x *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      // each row for itself: no other row's keys change its bits
      mx = mx > w.m[i] + kRescaleThreshold ? mx : w.m[i];
      const float a = weight(w.m[i], mx);
      w.m[i] = mx;
      w.neg_m[i] = mx == -INFINITY ? 0.f : __fsub_rn(0.f, mx);  // never -0
      w.raise_at[i] = (mx + kRescaleThreshold) / w.c[i];
      if (was_far || fabsf(w.neg_m[i]) >= kFarScore) {
        if (!was_far) w.c[i] *= 0x1p-24f;
        const float inv = rcp_approx(w.c[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) s[h][i] = __fadd_rn(__fmul_rn(s[h][i], w.c[i]) * 0x1p24f, w.neg_m[i]) * inv;
        w.neg_m[i] = -0.f;
        w.raise_at[i] = -INFINITY;
      }
      w.l[i] *= a;
#pragma unroll
      for (int G = 0; G < 4; ++G)
#pragma unroll
        for (int k = 0; k < 4; ++k) w.out(i, G, k) *= a;
    }
  }
  // ---- P^T, times V's scales per group, as operands with the keys along t
  uint32_t pb[C::kSums][C::kTiles][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float e[C::kMine];
#pragma unroll
    for (int i = 0; i < C::kMine; ++i) {
      e[i] = ex2_approx(fmaf(s[h][i], w.c[i], w.neg_m[i]));
      w.l[i] += e[i];
      e[i] *= w.up[i];
    }
    // a weight times a scale; what belongs to a hidden row may be anything
    auto product = [&](int i, int c) { return CUT && !seen[h][i] ? 0.f : e[i] * v_scale(h, c); };
#pragma unroll
    for (int c = 0; c < C::kSums; ++c)
#pragma unroll
      for (int nt = 0; nt < C::kTiles; ++nt)
        pb[c][nt][h] = transpose_8x8(
            C::kHalves ? pack_bf16x2(product(0, c), product(0, c + 2))
                       : pack_bf16x2(product(2 * nt, c), product(C::kMine > 1 ? 2 * nt + 1 : 0, c)));
  }
  // ---- O^T += V^T P^T
  if (ROWS != 8) load_v();
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t a[4][2];  // the group's four channels: rows 2t, 2t + 1 and 2t + 8, 2t + 9
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (BITS == 4) {
        const Fields v = v4_fields(vw[2 * h][c >> 1], vw[2 * h + 1][c >> 1], c);
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i][h] = v.pair(i);
      } else {
        const V8 v = {vw[2 * h][c % (2 * kWords)], vw[2 * h + 1][c % (2 * kWords)]};
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i][h] = v.pair(i);
      }
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int nt = 0; nt < C::kTiles; ++nt)
        mma_bf16(w.o[2 * c + f][nt], a[2 * f][0], a[2 * f + 1][0], a[2 * f][1], a[2 * f + 1][1],
                 pb[c % C::kSums][nt][0], pb[c % C::kSums][nt][1]);
  }
}

// The warps' parts of a tile.
template <int ROWS, int kWarps>
struct Parts {
  float O[kWarps][ROWS][kD];
  float M[kWarps][ROWS], L[kWarps][ROWS];
};

// Joins them; emit(r, M, L, a) gets row r, four channels a lane, from the warp that joined it.
template <int ROWS, int BITS, int kWarps, class Emit>
__device__ __forceinline__ void join_warps(Parts<ROWS, kWarps>& sm, State<ROWS, BITS>& w, int warp, int lane,
                                           Emit&& emit) {
  using C = Cols<ROWS>;
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < C::kMine; ++i) {
    const int r = C::row(i, t);
    const float down = w.down(i);
#pragma unroll
    for (int x = 4; x < 32; x *= 2) w.l[i] += __shfl_xor_sync(0xffffffffu, w.l[i], x);
    if (g == 0) {
      sm.M[warp][r] = w.m[i];
      sm.L[warp][r] = w.l[i];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<float4*>(&sm.O[warp][r][32 * c + 4 * g]) =
          make_float4(w.true_out(i, c, 0, down), w.true_out(i, c, 1, down), w.true_out(i, c, 2, down),
                      w.true_out(i, c, 3, down));
  }
  __syncthreads();
  for (int r = warp; r < ROWS; r += kWarps) {
    // lane x has part x's maximum and sum
    const float m = lane < kWarps ? sm.M[lane < kWarps ? lane : 0][r] : -INFINITY;
    float M = m;
#pragma unroll
    for (int x = 1; x < kWarps; x *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    M = __shfl_sync(0xffffffffu, M, 0);
    const float f = lane < kWarps ? weight(m, M) : 0.f;
    float L = lane < kWarps ? f * sm.L[lane < kWarps ? lane : 0][r] : 0.f;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) L += __shfl_xor_sync(0xffffffffu, L, x);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float fx = __shfl_sync(0xffffffffu, f, x);
      const float4 v = *reinterpret_cast<const float4*>(&sm.O[x][r][lane * 4]);
      a = make_float4(a.x + fx * v.x, a.y + fx * v.y, a.z + fx * v.z, a.w + fx * v.w);
    }
    emit(r, M, L, a);
  }
}

// ------------------------------------------------------------------ a cluster for each tile

// Few keys a warp: a ring of two units, 4.5 KB each, of each warp's own.
template <int BITS>
constexpr int unit_keys() { return BITS == 4 ? 32 : 16; }
constexpr int kUnits = 2;

template <int ROWS, int BITS, int kWarps>
struct ClusterSmem {
  uint8_t ring[kWarps][kUnits][unit_keys<BITS>() * cache_row_bytes(BITS)];
  Parts<ROWS, kWarps> parts;
  float cM[ROWS], cL[ROWS];
  uint64_t full[kWarps][kUnits];
  int abort;
};

constexpr int warps_per_sm(int ROWS) { return ROWS == 16 ? 12 : 16; }  // 168 and 128 registers a thread

template <int ROWS, int BITS, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, warps_per_sm(ROWS) / kWarps)
    cache_decode_kernel(const __grid_constant__ CacheDecode p) {
  constexpr int kKeys = unit_keys<BITS>(), kRec = cache_row_bytes(BITS);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<ClusterSmem<ROWS, BITS, kWarps>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % p.cluster;
  int tile = static_cast<int>(blockIdx.x) / p.cluster;
  const int mt = tile % p.row_tiles;
  tile /= p.row_tiles;
  uint64_t* full = sm.full[warp];
  if (lane == 0) {
    for (int i = 0; i < kUnits; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) sm.abort = 0;
  __syncthreads();
  const int b = tile / p.Hkv;
  const Tile a = make_tile(p, length(p, p.lens[b]), b, tile % p.Hkv, mt, ROWS, kKeys);
  const Share share(a.units, p.cluster * kWarps);
  const int me = rank * kWarps + warp;
  int u = share.begin(me);
  const int u1 = share.begin(me + 1);
  const uint8_t* head = p.cache + a.b * p.c_bs + a.hk * p.c_hs;
  auto fetch = [&](int x, int at) {  // by one lane
    const int j0 = first_key(a, x, kKeys);
    const uint32_t bytes = static_cast<uint32_t>(keys_of(a, x, j0, kKeys)) * kRec;
    mbar_arrive_expect_tx(&full[at], bytes);
    bulk_load(sm.ring[warp][at], head + static_cast<long long>(j0) * kRec, bytes, &full[at]);
  };
  const RawQ<ROWS> raw = load_q<ROWS>(p, a, g, t);
  if (lane == 0)
    for (int i = 0; i < kUnits && u + i < u1; ++i) fetch(u + i, i);
  State<ROWS, BITS> w;
  begin(w, raw, p, a, g, t);
  int at = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (; u < u1; ++u) {
    ok = mbar_wait_warp(&full[at], phase, &sm.abort, p.st, kWhere);
    if (!ok) break;
    const uint8_t* rec = sm.ring[warp][at];
    const int j0 = first_key(a, u, kKeys), nk = keys_of(a, u, j0, kKeys);
    if (u >= a.whole0 && u < a.whole1) {
#pragma unroll
      for (int i = 0; i < kKeys; i += kStep) step<ROWS, BITS, false>(w, p, rec + i * kRec, j0 + i, kStep, g, t);
    } else {
      for (int i = 0; i < nk; i += kStep) step<ROWS, BITS, true>(w, p, rec + i * kRec, j0 + i, nk - i, g, t);
    }
    __syncwarp();  // the unit has been read: its place is free
    if (lane == 0 && u + kUnits < u1) fetch(u + kUnits, at);
    at ^= 1;
    phase ^= static_cast<uint32_t>(at == 0);
  }
  if (!ok && lane == 0)  // copies in flight land before the CTA can end
    for (const int end = min(u + kUnits, u1); u < end; ++u) {
      drain_wait(&full[at], phase, p.st.limit);
      at ^= 1;
      phase ^= static_cast<uint32_t>(at == 0);
    }
  __syncwarp();
  join_warps(sm.parts, w, warp, lane, [&](int r, float M, float L, float4 v) {  // into slot 0
    *reinterpret_cast<float4*>(&sm.parts.O[0][r][4 * lane]) = v;
    if (lane == 0) {
      sm.cM[r] = M;
      sm.cL[r] = L;
    }
  });
  // ---- row r by rank r % cluster
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int r = rank + p.cluster * warp; r < ROWS; r += p.cluster * kWarps) {
    float M = -INFINITY;
    for (int c = 0; c < p.cluster; ++c) M = fmaxf(M, *cluster.map_shared_rank(&sm.cM[r], c));
    float L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < p.cluster; ++c) {
      const float f = weight(*cluster.map_shared_rank(&sm.cM[r], c), M);
      const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.parts.O[0][r][4 * lane], c));
      L += f * *cluster.map_shared_rank(&sm.cL[r], c);
      v = make_float4(v.x + f * x.x, v.y + f * x.y, v.z + f * x.z, v.w + f * x.w);
    }
    store_row(p, a, r, M, L, v, lane);
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// ------------------------------------------------------------------ the units of all tiles as one line
//
// (cache_line.cuh.) A CTA to an SM, whose warps take the sixteens of a unit: one
// bulk copy brings 16 keys for each, and its place is refilled once all have read
// it, so that the warps stay within a ring's length of one another (with a ring
// for each warp, or two CTAs to an SM, the scheduler lets some warps finish long
// before the others, which then run alone). Who refills: with a ring of four or
// more, a warp in turn, a unit later, by when the others mostly have read theirs
// too; with two there is no time to lose, and the last one to have read does it,
// as a counter tells (us, in turn / the last: 8 heads x 524288 keys in 4 bits 105 /
// 110; 8 x 131072 in 8 bits 66 / 51).

template <int ROWS, int BITS>
struct Line {
  static constexpr int kWarps = warps_per_sm(ROWS);
  static constexpr int kKeys = kWarps * kStep;                  // of a unit
  static constexpr int kBytes = kKeys * cache_row_bytes(BITS);
  static constexpr int kDepth = BITS == 4 ? 4 : 2;              // units of the ring
  static constexpr bool kInTurn = kDepth > 2;
  struct Smem {
    uint8_t ring[kDepth][kBytes];
    Parts<ROWS, kWarps> parts;
    uint64_t full[kDepth], empty[kDepth];
    int done[kDepth];  // warps that have read the unit in this place
    int abort;
    int lens[kLineSequences];
  };
};

__device__ __forceinline__ int add_acq_rel(int* at, int x) {
  int old;
  asm volatile("atom.acq_rel.cta.shared::cta.add.s32 %0, [%1], %2;" : "=r"(old) : "r"(smem_u32(at)), "r"(x) : "memory");
  return old;
}

template <int ROWS, int BITS>
__global__ void __launch_bounds__(32 * warps_per_sm(ROWS), 1)
    cache_decode_line_kernel(const __grid_constant__ CacheDecode p) {
  using F = Line<ROWS, BITS>;
  constexpr int kWarps = F::kWarps, kKeys = F::kKeys, kDepth = F::kDepth, kRec = cache_row_bytes(BITS);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<typename F::Smem*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int cta = static_cast<int>(blockIdx.x);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel waits for this one's end
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDepth; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
      sm.done[i] = 0;
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  copy_lengths(p, sm.lens);
  __syncthreads();
  Walk<ROWS, kKeys> walk;
  if (!walk.start(p, sm.lens, cta, static_cast<int>(gridDim.x), lane)) return;
  const Tile& a = walk.a;
  auto fetch = [&](int u, int at) {  // by one lane
    const uint8_t* head = p.cache + a.b * p.c_bs + a.hk * p.c_hs;
    const int j0 = first_key(a, u, kKeys);
    const uint32_t bytes = static_cast<uint32_t>(keys_of(a, u, j0, kKeys)) * kRec;
    mbar_arrive_expect_tx(&sm.full[at], bytes);
    bulk_load(sm.ring[at], head + static_cast<long long>(j0) * kRec, bytes, &sm.full[at]);
  };
  int n = walk.here();
  RawQ<ROWS> raw = load_q<ROWS>(p, a, g, t);
  if (threadIdx.x == 0)
    for (int i = 0; i < kDepth && i < n; ++i) fetch(walk.off + i, i);
  int at = 0;
  uint32_t phase = 0;
  bool ok = true;
  float* slot = p.workspace + 2LL * cta * slot_floats(ROWS);
  for (;;) {
    State<ROWS, BITS> w;
    begin(w, raw, p, a, g, t);
    const int end = walk.off + n;
    // the unit after which this warp refills
    int turn = walk.off + (warp + kWarps - (walk.off - 1 + kDepth) % kWarps) % kWarps;
    for (int u = walk.off; u < end; ++u) {
      ok = mbar_wait_warp(&sm.full[at], phase, &sm.abort, p.st, kWhere);
      if (!ok) break;
      const uint8_t* rec = sm.ring[at] + warp * kStep * kRec;
      if (u >= a.whole0 && u < a.whole1) {
        step<ROWS, BITS, false>(w, p, rec, 0, kStep, g, t);
      } else {
        const int j0 = first_key(a, u, kKeys), nk = keys_of(a, u, j0, kKeys) - warp * kStep;
        if (nk > 0) step<ROWS, BITS, true>(w, p, rec, j0 + warp * kStep, nk, g, t);
      }
      __syncwarp();
      if (F::kInTurn) {
        if (lane == 0) mbar_arrive(&sm.empty[at]);
        if (u == turn) {
          turn += kWarps;
          const int x = u - 1 + kDepth, back = at == 0 ? kDepth - 1 : at - 1;  // in the place of the unit before this one
          if (lane == 0 && u > walk.off && x < end &&
              mbar_wait_inline(&sm.empty[back], phase ^ static_cast<uint32_t>(at == 0), &sm.abort, p.st, kWhere + 0x10000u))
            fetch(x, back);
        }
      } else if (lane == 0 && add_acq_rel(&sm.done[at], 1) == kWarps - 1) {
        sm.done[at] = 0;
        if (u + kDepth < end) fetch(u + kDepth, at);
      }
      if (++at == kDepth) {
        at = 0;
        phase ^= 1u;
      }
    }
    const Tile now = a;
    const bool whole = n == a.units;
    walk.advance(p, sm.lens, n);
    __syncthreads();  // the ring is empty, or a wait ran out
    if (sm.abort) break;
    if (walk.left > 0) {  // the next tile's copies are on their way while this one's parts are joined
      n = walk.here();
      raw = load_q<ROWS>(p, a, g, t);
      if (threadIdx.x == 0)
        for (int i = 0, x = at; i < kDepth && i < n; ++i, x = x + 1 == kDepth ? 0 : x + 1) fetch(walk.off + i, x);
    }
    join_warps(sm.parts, w, warp, lane, [&](int r, float M, float L, float4 v) {
      if (whole) {
        store_row(p, now, r, M, L, v, lane);
      } else {
        *reinterpret_cast<float4*>(slot + r * kD + 4 * lane) = v;
        if (lane == 0) {
          slot[ROWS * kD + r] = M;
          slot[ROWS * (kD + 1) + r] = L;
        }
      }
    });
    if (walk.left <= 0) break;
    slot = p.workspace + (2LL * cta + 1) * slot_floats(ROWS);
  }
  if (!ok && threadIdx.x == 0)  // copies in flight land before the CTA ends
    for (int i = 0; i < kDepth; ++i) {
      drain_wait(&sm.full[at], phase, p.st.limit);
      if (++at == kDepth) {
        at = 0;
        phase ^= 1u;
      }
    }
}
// ------------------------------------------------------------------ launches

template <int ROWS, int BITS, int kWarps>
struct ClusterForm {
  static constexpr int kSmem = sizeof(ClusterSmem<ROWS, BITS, kWarps>);
  static const void* fn() { return reinterpret_cast<const void*>(cache_decode_kernel<ROWS, BITS, kWarps>); }

  static DeviceOnce& allowed() {
    static DeviceOnce once;
    return once;
  }

  static int resident(const ContextKey& at, int cluster) {
    static ClusterCounts known;
    return resident_clusters(known, at, allowed(), fn(), 32 * kWarps, kSmem, cluster);
  }

  // The largest cluster with which all tiles are resident at once, every warp having a unit; 0 if none.
  static int one_wave(const ContextKey& at, long long tiles, long long units) {
    for (int c = static_cast<int>(std::min<long long>(kMaxCluster, std::max<long long>(1, units / kWarps))); c > 0; --c)
      if (resident(at, c) >= tiles) return c;
    return 0;
  }

  static int launch(const CacheDecode& p, long long tiles, cudaStream_t stream) {
    const int rc = allow_clusters_once(allowed(), fn(), kSmem);
    if (rc != 0) return rc;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(p.cluster);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_decode_kernel<ROWS, BITS, kWarps>, p) == cudaSuccess ? 0 : -4;
  }
};

template <int ROWS, int BITS>
struct LineForm {
  static constexpr int kSmem = sizeof(typename Line<ROWS, BITS>::Smem), kThreads = 32 * Line<ROWS, BITS>::kWarps;
  static const void* fn() { return reinterpret_cast<const void*>(cache_decode_line_kernel<ROWS, BITS>); }

  static DeviceOnce& allowed() {
    static DeviceOnce once;
    return once;
  }

  static int ctas(const ContextKey& at) {  // that the GPU holds at once
    static ClusterCounts known;
    return resident_clusters(known, at, allowed(), fn(), kThreads, kSmem, 1);
  }

  static size_t workspace(int n) { return 2 * sizeof(float) * slot_floats(ROWS) * static_cast<size_t>(n); }

  static int launch(const CacheDecode& p, long long tiles, int n, cudaStream_t stream) {
    const int rc = allow_clusters_once(allowed(), fn(), kSmem);
    if (rc != 0) return rc;
    cache_decode_line_kernel<ROWS, BITS><<<n, kThreads, kSmem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return -4;
    return launch_cache_join<ROWS, Line<ROWS, BITS>::kKeys>(p, tiles, n, stream);
  }
};

// Sizes of a call as its launch sees them: the host knows no lengths.
struct Plan {
  int B, rows;
  long long row_tiles, tiles, keys;  // keys: the most that a tile can see
};

Plan plan_of(int B, int H, int Hkv, int T, int Smax, int window, int sinks) {
  Plan a;
  a.B = B;
  const long long R = static_cast<long long>(T) * (H / Hkv);
  a.rows = R <= 4 ? 4 : R <= 8 ? 8 : 16;
  a.row_tiles = (R + a.rows - 1) / a.rows;
  a.tiles = static_cast<long long>(B) * Hkv * a.row_tiles;
  a.keys = std::min<long long>(Smax, static_cast<long long>(window) + T - 1 + sinks);
  return a;
}

// The cluster form of a call: 4 or 8 warps a CTA, whichever puts more warps on
// the GPU in one wave, and the cluster (1 where not even that fits).
template <int ROWS, int BITS>
struct ClusterChoice {
  int warps, cluster;
  long long all_warps;  // of the tiles
  ClusterChoice(const Plan& a, const ContextKey& at) {
    const long long units = (a.keys + unit_keys<BITS>() - 1) / unit_keys<BITS>();
    const int c4 = ClusterForm<ROWS, BITS, 4>::one_wave(at, a.tiles, units);
    const int c8 = ROWS == 16 ? 0 : ClusterForm<ROWS, BITS, 8>::one_wave(at, a.tiles, units);
    warps = 4 * c4 >= 8 * c8 ? 4 : 8;
    cluster = std::max(1, warps == 4 ? c4 : c8);
    all_warps = a.tiles * cluster * warps;
  }
};

// CTAs of the line form, or 0 for the cluster form: two estimates in us, by the
// most keys that the sizes allow, fitted to both forms at fourteen sizes. A
// cluster form is done when its warps' share of the bytes is; the line form has a
// longer start, a second kernel, and some 3 us for each tile that a CTA begins
// after its first; with more than four rows it is bound by its instructions. us,
// cluster / line, 4 bits unless said: 32 heads x 2052 keys 8 / 10; 8 x 8 heads x
// 20001, eight rows, 38 / 42; 160 x 32772 127 / 114; 8 x 131072 in 8 bits 69 / 50; 8 x
// 524288 204 / 99; 1 x 524288 123 / 25; 4 x 100000 33 / 23; 512 x 2000 26 / 36; 80 x
// 5000 in 8 bits 20 / 24; 40 x 32768 40 / 38; 8 x 65536, eight rows 37 / 26, sixteen
// 56 / 37.
template <int ROWS, int BITS>
int line_ctas(const Plan& a, const ClusterChoice<ROWS, BITS>& c, const ContextKey& at) {
  const int n = LineForm<ROWS, BITS>::ctas(at);
  const long long units = a.tiles * ((a.keys + Line<ROWS, BITS>::kKeys - 1) / Line<ROWS, BITS>::kKeys + 1);
  if (n <= 0 || a.B > kLineSequences || a.row_tiles > 8 || units + a.tiles * kTileCost<ROWS> >= 1LL << 31) return 0;
  const double hbm_us = static_cast<double>(a.tiles) * a.keys * cache_row_bytes(BITS) / 6.7e6;
  const double busy = std::min(1.0, static_cast<double>(c.all_warps) / (n * warps_per_sm(ROWS)));  // n: one CTA to an SM
  const double cluster_us = 5 + 1.15 * hbm_us / std::min(1.0, (BITS == 4 ? 1.0 : 1.5) * busy);
  const double more = std::max(0.0, static_cast<double>(a.tiles) / n - 1);
  const double line_us = 12 + (BITS == 4 && ROWS > 4 ? 1.25 : 1.08) * hbm_us + 3.5 * more;
  return line_us < cluster_us ? n : 0;
}

template <int ROWS, int BITS>
int launch_rows(CacheDecode& p, const Plan& a, size_t ws_bytes, cudaStream_t stream) {
  const ContextKey at = current_context();
  const ClusterChoice<ROWS, BITS> c(a, at);
  const int n = line_ctas<ROWS, BITS>(a, c, at);
  if (n > 0) {
    if (!p.workspace || ws_bytes < LineForm<ROWS, BITS>::workspace(n)) return -1;
    return LineForm<ROWS, BITS>::launch(p, a.tiles, n, stream);
  }
  p.cluster = c.cluster;
  return c.warps == 4 ? ClusterForm<ROWS, BITS, 4>::launch(p, a.tiles, stream)
                      : ClusterForm<ROWS, BITS, 8>::launch(p, a.tiles, stream);
}

// f with the row count and the bits as types.
template <class F>
auto with_form(int rows, int bits, F&& f) {
  if (bits == 4)
    return rows == 4   ? f.template operator()<4, 4>()
           : rows == 8 ? f.template operator()<8, 4>()
                       : f.template operator()<16, 4>();
  return rows == 4   ? f.template operator()<4, 8>()
         : rows == 8 ? f.template operator()<8, 8>()
                     : f.template operator()<16, 8>();
}

struct WorkspaceOf {
  const Plan& a;
  template <int ROWS, int BITS>
  size_t operator()() const {
    const ContextKey at = current_context();
    return LineForm<ROWS, BITS>::workspace(line_ctas<ROWS, BITS>(a, ClusterChoice<ROWS, BITS>(a, at), at));
  }
};

struct Launch {
  CacheDecode& p;
  const Plan& a;
  size_t ws_bytes;
  cudaStream_t stream;
  template <int ROWS, int BITS>
  int operator()() const {
    return launch_rows<ROWS, BITS>(p, a, ws_bytes, stream);
  }
};

}  // namespace

// CTAs of the form with 128-row tiles (attn_cache_tiles.cu), or 0 for one of the
// forms here, which unpack the keys once for every sixteen rows: two estimates in
// us. us, those here / 128-row tiles: 8 heads x 65536 keys, 32 rows 61 / 49, 64 rows
// 104 / 50, in 8 bits 131 / 62; 32 x 20000, 128 rows 201 / 59; 8 x 65536, window 16384,
// 4000 rows 1237 / 357; 8 x 2000, 56 rows 13 / 17; 8 x 500, 20 rows 10 / 14.
static int tiles_ctas(const Plan& a, int T, int G, int bits, const ContextKey& at) {
  const long long R = static_cast<long long>(T) * G;
  if (R <= 16 || a.B > kLineSequences) return 0;
  const long long units = a.tiles / a.row_tiles * ((R + 127) / 128) * (a.keys / 128 + 2);
  if (units + a.tiles * kTileCost<128> >= 1LL << 31) return 0;
  const int n = cache_tiles_ctas(bits, at);
  if (n <= 0) return 0;
  const double tiles_us = 12 + (bits == 4 ? 1.3 : 1.7) * static_cast<double>(units) / n;
  const double here_us = 9 + 0.75e-3 * static_cast<double>(a.tiles) * ((a.keys + 15) / 16);
  return tiles_us < here_us ? n : 0;
}

size_t cache_decode_workspace(int B, int H, int Hkv, int T, int Smax, int window, int sinks, int bits) {
  const Plan a = plan_of(B, H, Hkv, T, Smax, window, sinks);
  const int n = tiles_ctas(a, T, H / Hkv, bits, current_context());
  if (n > 0) return cache_tiles_workspace(n);
  return with_form(a.rows, bits, WorkspaceOf{a});
}

int cache_decode_form(int B, int H, int Hkv, int T, int Smax, int window, int sinks, int bits) {
  const Plan a = plan_of(B, H, Hkv, T, Smax, window, sinks);
  if (tiles_ctas(a, T, H / Hkv, bits, current_context()) > 0) return LCB_CACHE_FORM_TILES;
  return cache_decode_workspace(B, H, Hkv, T, Smax, window, sinks, bits) ? LCB_CACHE_FORM_LINE : LCB_CACHE_FORM_CLUSTER;
}

int launch_cache_decode(CacheDecode p, int bits, size_t ws_bytes, cudaStream_t stream) {
  p.G = p.H / p.Hkv;
  if (static_cast<long long>(p.T) * p.G > kWindowMaxRows) return -1;
  const Plan a = plan_of(p.B, p.H, p.Hkv, p.T, p.Smax, p.window, p.sinks);
  if (a.tiles > 0x7fffffffLL / kMaxCluster) return -1;
  const int n = tiles_ctas(a, p.T, p.G, bits, current_context());
  if (n > 0)
    return p.workspace && ws_bytes >= cache_tiles_workspace(n) ? launch_cache_tiles(p, bits, n, stream) : -1;
  p.row_tiles = static_cast<int>(a.row_tiles);
  p.cluster = 1;
  return with_form(a.rows, bits, Launch{p, a, ws_bytes, stream});
}

}  // namespace lcb
