// Attention of the newest tokens over a quantised K/V cache (kv_cache.cuh),
// with the mask of the windowed attention: the query at position p sees keys
// j <= p with p - j < window, and the first `sinks` keys.
//
// A cached row holds, per group G of 32 channels, whole numbers and a scale:
//   k_jc = s^K_jG n_jc,   x_ij = scale * sum_G s^K_jG sum_{c in G} q_ic n_jc
//   v_jc = s^V_jG n_jc,   o_ic = sum_j (p_ij s^V_jG) n_jc / l_i
// so the products take the whole numbers, which bf16 holds exactly, and the
// scales go to the scores and to the weights: nothing of the cache is rounded.
// (p s^V is rounded to bf16 for the second product, as P is in the other
// forms: half a step, up to 2^-8 of each weight, of either sign.)
//
// Every visible record (144 or 272 bytes) is read once for all query rows that
// share its head, up to 16 of them. HBM bounds it only if little is done per
// byte: at 6.7 TB/s an SM gets a key every 6 clocks (4 bits), 24 issue slots
// for its 256 numbers. Hence
//   S^T[16 keys][8 rows] = K Q^T  and  O^T[128][8 rows] += V^T P^T  on warp
//     mma.sync (m16n8k16) with operands in registers, as attn_window_split.cu:
//     tcgen05 would want its operand unpacked into shared or tensor memory;
//   codes stored in operand order, so that a shift, one bitwise operation and a
//     packed add make two of them bf16 numbers;
//   records brought to shared memory by bulk copies, one instruction for a
//     unit of 4.5 KB, in a ring of each warp's own: no address arithmetic and
//     no barrier among warps.
//
// The visible keys of a (sequence, K/V head, row tile) are split evenly over
// the warps of a cluster of CTAs, whose partial (m, l, O) are joined in shared
// memory, then through distributed shared memory. Where there are too few
// tiles for clusters to fill the GPU, a tile gets several clusters, which leave
// partials in a workspace for a second kernel. No atomics: the same result
// every time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attn_window.cuh"
#include "kv_cache.cuh"
#include "lcb_internal.h"
#include "mma_warp.cuh"

namespace cg = cooperative_groups;

namespace lcb {
namespace {

constexpr int kD = 128;
constexpr int kStep = 16;   // keys of a product
constexpr int kDepth = 3;   // units of a warp's ring
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: the running maximum is raised lazily, P stays <= 256
constexpr uint32_t kWhere = 9u << 24;

template <int BITS>
struct Unit {  // keys that one bulk copy brings
  static constexpr int kKeys = BITS == 4 ? 32 : 16;
  static constexpr int kBytes = kKeys * cache_row_bytes(BITS);
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Contiguous bytes (a multiple of 16, both ends aligned to 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Weight of a partial with maximum m in a sum with maximum M >= m (both -inf: the partial is empty, or NaN).
__device__ __forceinline__ float weight(float m, float M) { return m == M ? 1.f : ex2_approx(m - M); }

// A CTA's shared memory. The ring's bytes become the warps' partials, joined into slot 0, once the keys are done.
template <int NT, int BITS, int kWarps>
struct Smem {
  static constexpr int kRows = 8 * NT;
  union {
    uint8_t ring[kWarps][kDepth][Unit<BITS>::kBytes];
    float O[kWarps][kRows][kD];
  };
  float M[kWarps][kRows], L[kWarps][kRows];
  float cM[kRows], cL[kRows];
  uint64_t full[kWarps][kDepth];
  int abort;
};

// NT: 8-row tiles of query rows (1 or 2); kWarps: warps of a CTA.
template <int NT, int BITS, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (NT == 1 ? 16 : 12) / kWarps) cache_decode_kernel(const __grid_constant__ CacheDecode p) {
  constexpr int kRows = 8 * NT;
  constexpr int kRec = cache_row_bytes(BITS), kPlanes = cache_planes(BITS);
  constexpr int kKeys = Unit<BITS>::kKeys;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<Smem<NT, BITS, kWarps>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % p.cluster;
  int tile = static_cast<int>(blockIdx.x) / p.cluster;
  const int part = tile % p.parts;
  tile /= p.parts;
  const int mt = tile % p.row_tiles;
  tile /= p.row_tiles;
  const int hk = tile % p.Hkv, b = tile / p.Hkv;
  const int G = p.H / p.Hkv, R = p.T * G;
  const int r0 = mt * kRows;  // rows r = (token r / G, query head hk * G + r % G)

  uint64_t* full = sm.full[warp];
  if (lane == 0) {
    for (int i = 0; i < kDepth; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) sm.abort = 0;
  __syncthreads();

  const int len = min(max(p.lens[b], 0), p.Smax);
  const int p0 = len - p.T;  // position of token 0
  const int p_min = p0 + r0 / G, p_max = p0 + min(R - 1, r0 + kRows - 1) / G;
  // keys that a row of this tile sees: [0, ns) and [lo, hi), in units that do not cross from one to the other
  const int lo = max(0, p_min - p.window + 1), hi = min(len, p_max + 1);
  const int ns = max(0, min(min(p.sinks, lo), hi));
  const int sink_units = (ns + kKeys - 1) / kKeys;
  const int units = sink_units + (max(0, hi - lo) + kKeys - 1) / kKeys;
  auto first_key = [&](int u) { return u < sink_units ? u * kKeys : lo + (u - sink_units) * kKeys; };
  auto keys_of = [&](int u) { return min(kKeys, (u < sink_units ? ns : hi) - first_key(u)); };

  // this warp's units
  const long long workers = static_cast<long long>(p.parts) * p.cluster * kWarps;
  const long long me = (static_cast<long long>(part) * p.cluster + rank) * kWarps + warp;
  const int u0 = static_cast<int>(me * units / workers), u1 = static_cast<int>((me + 1) * units / workers);

  const uint8_t* head = p.cache + b * p.c_bs + hk * p.c_hs;
  uint8_t(*ring)[Unit<BITS>::kBytes] = sm.ring[warp];
  auto fetch = [&](int u, int at) {  // lane 0
    const uint32_t bytes = static_cast<uint32_t>(keys_of(u)) * kRec;
    mbar_arrive_expect_tx(&full[at], bytes);
    bulk_load(ring[at], head + static_cast<long long>(first_key(u)) * kRec, bytes, &full[at]);
  };
  if (lane == 0)
    for (int i = 0; i < kDepth && u0 + i < u1; ++i) fetch(u0 + i, i);

  // Q fragments, in K's channel order
  uint32_t qf[NT][8][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = r0 + 8 * nt + g;
    const __nv_bfloat16* src =
        p.q + b * p.q_bs + static_cast<long long>(r / G) * p.q_rs + (hk * G + r % G) * kD + 8 * t;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 v = r < R ? *reinterpret_cast<const uint4*>(src + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
      qf[nt][2 * c][0] = v.x;
      qf[nt][2 * c][1] = v.y;
      qf[nt][2 * c + 1][0] = v.z;
      qf[nt][2 * c + 1][1] = v.w;
    }
  }
  int pr[NT][2];  // positions of this lane's score columns (rows past the last see nothing)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * nt + 2 * t + e;
      pr[nt][e] = r < R ? p0 + r / G : -1;
    }

  float o[8][NT][4];  // o[2 c + f]: channels 32 c + 4 g + 2 f + {0, 1} of rows 2t, 2t + 1
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }

  int at = 0;
  uint32_t phase = 0;
  bool ok = true;
  int u = u0;
  for (; u < u1; ++u) {
    ok = mbar_wait_warp(&full[at], phase, &sm.abort, p.st, kWhere);
    if (!ok) break;
    const int j0 = first_key(u), nk = keys_of(u);
    // every key of the unit is seen by every row of the tile
    const bool whole = nk == kKeys && j0 + kKeys - 1 <= p_min && (p_max - j0 < p.window || j0 + kKeys <= p.sinks);
#pragma unroll
    for (int sub = 0; sub < kKeys / kStep; ++sub) {
      if (sub * kStep >= nk) break;
      const uint8_t* rec = ring[at] + sub * kStep * kRec;
      // scales of keys g and g + 8: four of K, four of V
      const uint4 sc[2] = {*reinterpret_cast<const uint4*>(rec + g * kRec + cache_scale_offset(BITS)),
                           *reinterpret_cast<const uint4*>(rec + (g + 8) * kRec + cache_scale_offset(BITS))};
      // ---- S^T: s[nt][2u + e] is key 8u + g, row 8 nt + 2t + e
      float s[NT][4];
      {
        uint4 kw[kPlanes][2];
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            kw[pl][h] = *reinterpret_cast<const uint4*>(rec + (g + 8 * h) * kRec + pl * kPlaneBytes + 16 * t);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
          uint32_t w[kPlanes][2];
#pragma unroll
          for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[pl][h] = c == 0 ? kw[pl][h].x : c == 1 ? kw[pl][h].y : c == 2 ? kw[pl][h].z : kw[pl][h].w;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a0 = codes_bf16x2<BITS>(w[0][0], w[kPlanes - 1][0], 2 * h);
            const uint32_t a1 = codes_bf16x2<BITS>(w[0][1], w[kPlanes - 1][1], 2 * h);
            const uint32_t a2 = codes_bf16x2<BITS>(w[0][0], w[kPlanes - 1][0], 2 * h + 1);
            const uint32_t a3 = codes_bf16x2<BITS>(w[0][1], w[kPlanes - 1][1], 2 * h + 1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(acc[nt], a0, a1, a2, a3, qf[nt][2 * c + h][0], qf[nt][2 * c + h][1]);
          }
          const uint32_t k0 = c < 2 ? sc[0].x : sc[0].y, k1 = c < 2 ? sc[1].x : sc[1].y;
          const float s0 = c & 1 ? bf16hi_to_f32(k0) : bf16lo_to_f32(k0);
          const float s1 = c & 1 ? bf16hi_to_f32(k1) : bf16lo_to_f32(k1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f = e < 2 ? s0 : s1;
              s[nt][e] = c == 0 ? f * acc[nt][e] : fmaf(f, acc[nt][e], s[nt][e]);
            }
        }
      }
      bool seen[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] *= p.scale_log2;
      if (!whole) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int i = sub * kStep + 8 * h + g, j = j0 + i;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int pp = pr[nt][e];
              seen[nt][2 * h + e] = i < nk && j <= pp && (pp - j < p.window || j < p.sinks);
              if (!seen[nt][2 * h + e]) s[nt][2 * h + e] = -INFINITY;
            }
        }
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) raise |= s[nt][e] > m[nt][e & 1] + kRescaleThreshold;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[nt][e], s[nt][2 + e]);
#pragma unroll
            for (int w = 4; w < 32; w *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            // each row for itself: no other row's keys change its bits
            mx = mx > m[nt][e] + kRescaleThreshold ? mx : m[nt][e];
            const float a = weight(m[nt][e], mx);
            m[nt][e] = mx;
            l[nt][e] *= a;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][nt][e] *= a;
              o[i][nt][2 + e] *= a;
            }
          }
      }
      // ---- P^T, times V's scales per group, as operands with the keys along t
      uint32_t pb[NT][4][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float e0 = ex2_approx(s[nt][2 * h] - m0), e1 = ex2_approx(s[nt][2 * h + 1] - m1);
          l[nt][0] += e0;
          l[nt][1] += e1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t w = c < 2 ? sc[h].z : sc[h].w;
            const float f = c & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
            float x0 = e0 * f, x1 = e1 * f;
            if (!whole) {  // a hidden row's scale may be anything
              x0 = seen[nt][2 * h] ? x0 : 0.f;
              x1 = seen[nt][2 * h + 1] ? x1 : 0.f;
            }
            pb[nt][c][h] = transpose_8x8(pack_bf16x2(x0, x1));
          }
        }
      }
      // ---- O^T += V^T P^T
      uint2 vw[kPlanes][4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          vw[pl][i] = *reinterpret_cast<const uint2*>(rec + (2 * t + (i & 1) + 8 * (i >> 1)) * kRec +
                                                      cache_v_offset(BITS) + pl * kPlaneBytes + 8 * g);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t sel = c & 1 ? 0x7632 : 0x5410;
        uint32_t x[kPlanes][2];  // a channel's codes of two keys, 16 bits apart
#pragma unroll
        for (int pl = 0; pl < kPlanes; ++pl)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            x[pl][h] = c < 2 ? __byte_perm(vw[pl][2 * h].x, vw[pl][2 * h + 1].x, sel)
                             : __byte_perm(vw[pl][2 * h].y, vw[pl][2 * h + 1].y, sel);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const uint32_t a0 = codes_bf16x2<BITS>(x[0][0], x[kPlanes - 1][0], 2 * f);
          const uint32_t a1 = codes_bf16x2<BITS>(x[0][0], x[kPlanes - 1][0], 2 * f + 1);
          const uint32_t a2 = codes_bf16x2<BITS>(x[0][1], x[kPlanes - 1][1], 2 * f);
          const uint32_t a3 = codes_bf16x2<BITS>(x[0][1], x[kPlanes - 1][1], 2 * f + 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816(o[2 * c + f][nt], a0, a1, a2, a3, pb[nt][c][0], pb[nt][c][1]);
        }
      }
    }
    __syncwarp();  // the unit has been read: its place is free
    if (lane == 0 && u + kDepth < u1) fetch(u + kDepth, at);
    if (++at == kDepth) {
      at = 0;
      phase ^= 1u;
    }
  }
  if (!ok && lane == 0)  // copies in flight land before the ring is used for anything else
    for (int i = u; i < min(u + kDepth, u1); ++i) {
      const int a = (i - u0) % kDepth;
      drain_wait(&full[a], static_cast<uint32_t>((i - u0) / kDepth) & 1u, p.st.limit);
    }
  __syncthreads();

  // ---- join the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * t + e;
#pragma unroll
      for (int w = 4; w < 32; w *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
      if (g == 0) {
        sm.M[warp][r] = m[nt][e];
        sm.L[warp][r] = l[nt][e];
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<float4*>(&sm.O[warp][r][32 * c + 4 * g]) =
            make_float4(o[2 * c][nt][e], o[2 * c][nt][2 + e], o[2 * c + 1][nt][e], o[2 * c + 1][nt][2 + e]);
    }
  __syncthreads();
  const int d4 = lane * 4;
  for (int r = warp; r < kRows; r += kWarps) {  // a warp joins a row: its partials into slot 0
    float M = sm.M[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm.M[w][r]);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight(sm.M[w][r], M);
      const float4 v = *reinterpret_cast<const float4*>(&sm.O[w][r][d4]);
      L += f * sm.L[w][r];
      a = make_float4(a.x + f * v.x, a.y + f * v.y, a.z + f * v.z, a.w + f * v.w);
    }
    *reinterpret_cast<float4*>(&sm.O[0][r][d4]) = a;
    if (lane == 0) {
      sm.cM[r] = M;
      sm.cL[r] = L;
    }
  }
  // ---- join the cluster: row r by rank r % cluster
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int r = rank + p.cluster * warp; r < kRows; r += p.cluster * kWarps) {
    if (r0 + r >= R) break;
    float M = -INFINITY;
    for (int c = 0; c < p.cluster; ++c) M = fmaxf(M, *cluster.map_shared_rank(&sm.cM[r], c));
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < p.cluster; ++c) {
      const float f = weight(*cluster.map_shared_rank(&sm.cM[r], c), M);
      const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sm.O[0][r][d4], c));
      L += f * *cluster.map_shared_rank(&sm.cL[r], c);
      a = make_float4(a.x + f * v.x, a.y + f * v.y, a.z + f * v.z, a.w + f * v.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int tok = (r0 + r) / G, h = hk * G + (r0 + r) % G;
    uint2 w;
    w.x = pack_bf16x2(a.x * inv, a.y * inv);
    w.y = pack_bf16x2(a.z * inv, a.w * inv);
    *reinterpret_cast<uint2*>(p.o + b * p.o_bs + static_cast<long long>(tok) * p.o_rs + h * kD + d4) = w;
    if (lane == 0)
      p.lse[b * p.l_bs + h * p.l_hs + tok] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

template <int NT, int BITS, int kWarps>
struct Form {
  static constexpr int kSmem = sizeof(Smem<NT, BITS, kWarps>);
  static const void* fn() { return reinterpret_cast<const void*>(cache_decode_kernel<NT, BITS, kWarps>); }

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
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.parts * p.cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_decode_kernel<NT, BITS, kWarps>, p) == cudaSuccess ? 0 : -4;
  }
};

template <int NT, int BITS>
int launch_rows(CacheDecode& p, long long tiles, long long units, cudaStream_t stream) {
  const ContextKey at = current_context();
  const int c4 = Form<NT, BITS, 4>::one_wave(at, tiles, units), c8 = Form<NT, BITS, 8>::one_wave(at, tiles, units);
  if (4 * c4 >= 8 * c8) {
    p.cluster = std::max(1, c4);
    return Form<NT, BITS, 4>::launch(p, tiles, stream);
  }
  p.cluster = c8;
  return Form<NT, BITS, 8>::launch(p, tiles, stream);
}

}  // namespace

size_t cache_decode_workspace(int, int, int, int, int, int, int, int) { return 0; }

int launch_cache_decode(CacheDecode p, int bits, size_t, cudaStream_t stream) {
  const long long R = static_cast<long long>(p.T) * (p.H / p.Hkv);
  if (R > kWindowMaxRows) return -1;
  const int rows = R <= 8 ? 8 : 16;
  p.row_tiles = static_cast<int>((R + rows - 1) / rows);
  p.parts = 1;
  const long long tiles = static_cast<long long>(p.B) * p.Hkv * p.row_tiles;
  if (tiles > 0x7fffffffLL / kMaxCluster) return -1;
  if (tiles == 0) return 0;
  // Most keys that a row tile can see, from the host's side of the sizes.
  const long long seen = std::min<long long>(p.Smax, static_cast<long long>(p.window) + p.T - 1 + p.sinks);
  const int keys = bits == 4 ? Unit<4>::kKeys : Unit<8>::kKeys;
  const long long units = (seen + keys - 1) / keys;
  if (bits == 4) return rows == 8 ? launch_rows<1, 4>(p, tiles, units, stream) : launch_rows<2, 4>(p, tiles, units, stream);
  return rows == 8 ? launch_rows<1, 8>(p, tiles, units, stream) : launch_rows<2, 8>(p, tiles, units, stream);
}

}  // namespace lcb
