// Windowed attention for few query rows per K/V head (the newest token or
// tokens of a sequence against its cache): exact softmax attention in which
// the query at position p sees keys j <= p with p - j < window, and the first
// `sinks` keys.
//
// Every visible K and V row is read once for all query rows that share its
// head; per key that is 512 bytes against 4 * 128 flops a row, so HBM bounds
// it for any number of rows up to the tile's 16 and the tensor work (warp
// mma.sync, M = 16 keys) hides under the loads. tcgen05 tiles would want 128
// query rows, of which a token supplies T * H / Hkv; and they would read K and
// V through shared memory, where here they go straight to registers.
//
//   S^T[16 keys][8 rows] = K Q^T  and  O^T[128][8 rows] += V^T P^T, m16n8k16.
//
// The sum over features and the order of O's features are free to permute, so
// each lane's 16-byte loads of K and V are operand fragments as they arrive:
//   K: lane (g, t) reads features 32c + 8t .. + 7 of keys g and g + 8, two
//      k-steps' A fragments; Q is laid out with the same permutation;
//   V: lane (g, t) reads features 64h + 8g .. + 7 of keys 2t, 2t+1, 2t+8,
//      2t+9; byte permutes pair the keys of a feature into A fragments.
// P^T leaves the first product with keys along g and rows along t; the second
// wants them exchanged, which movmatrix does on 8 x 8 blocks.
//
// The visible keys of a (sequence, K/V head) are split over a cluster of CTAs
// and their warps; partial (m, l, O) are joined in shared memory, then across
// the cluster through distributed shared memory: one launch, no workspace, no
// atomics, and the same result every time.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attn_window.cuh"
#include "lcb_internal.h"

namespace cg = cooperative_groups;

namespace lcb {
namespace {

constexpr int kD = 128;
constexpr int kSms = 152;
constexpr int kKeys = 16;  // keys per warp step
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units: the running maximum is raised lazily, P stays <= 256

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

__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Weight of a partial with maximum m in a sum with maximum M >= m (both -inf: the partial is empty, or NaN).
__device__ __forceinline__ float weight(float m, float M) { return m == M ? 1.f : ex2_approx(m - M); }

// A CTA's shared memory: its warps' partials, joined into slot 0, cM and cL.
template <int kRows, int kWarps>
struct Partials {
  float O[kWarps][kRows][kD];
  float M[kWarps][kRows], L[kWarps][kRows];
  float cM[kRows], cL[kRows];
};

// NT: 8-row tiles of query rows (1 or 2); kWarps: warps of a CTA.
template <int NT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) window_split_kernel(const __grid_constant__ WindowSplit p) {
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& [sO, sM, sL, cM, cL] = *reinterpret_cast<Partials<kRows, kWarps>*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(blockIdx.x) % p.cluster;
  int tile = static_cast<int>(blockIdx.x) / p.cluster;
  const int mt = tile % p.row_tiles;
  tile /= p.row_tiles;
  const int hk = tile % p.Hkv, b = tile / p.Hkv;
  const int G = p.H / p.Hkv, R = p.T * G;
  const int r0 = mt * kRows;  // rows r = (token r / G, query head hk * G + r % G)

  const int len = p.lens ? min(max(p.lens[b], 0), p.Sk) : p.Sk;
  const int p0 = p.lens ? len - p.T : p.pos0;  // position of token 0
  const int p_min = p0 + r0 / G, p_max = p0 + min(R - 1, r0 + kRows - 1) / G;
  // keys that a row of this tile sees: [0, ns) and [lo, hi)
  const int lo = max(0, p_min - p.window + 1), hi = min(len, p_max + 1);
  const int ns = max(0, min(min(p.sinks, lo), hi));
  const int n = ns + max(0, hi - lo);

  // Q fragments, in K's feature order
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

  const __nv_bfloat16* kb = p.k + b * p.kv_bs + hk * kD;
  const __nv_bfloat16* vb = p.v + b * p.kv_bs + hk * kD;
  const long long krs = p.kv_rs;
  auto key_of = [&](int i) { return i < ns ? i : i - ns + lo; };
  uint4 kf[2][4], vf[4][2];
  auto load_k = [&](int i0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + 8 * u + g;
      const __nv_bfloat16* src = kb + key_of(i) * krs + 8 * t;
#pragma unroll
      for (int c = 0; c < 4; ++c) kf[u][c] = i < n ? load16(src + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto load_v = [&](int i0) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 2 * t + (u & 1) + 8 * (u >> 1);
      const __nv_bfloat16* src = vb + key_of(i) * krs + 8 * g;
#pragma unroll
      for (int h = 0; h < 2; ++h) vf[u][h] = i < n ? load16(src + 64 * h) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  float o[8][NT][4];
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

  // this CTA's steps of 16 keys, dealt to its warps
  const int steps = (n + kKeys - 1) / kKeys;
  const int per = (steps + p.cluster - 1) / p.cluster;
  const int end = min(steps, (rank + 1) * per);
  int step = rank * per + warp;
  if (step < end) {
    load_k(step * kKeys);
    load_v(step * kKeys);
  }
  for (; step < end; step += kWarps) {
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816(s[nt], kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, qf[nt][2 * c][0], qf[nt][2 * c][1]);
        mma_16816(s[nt], kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, qf[nt][2 * c + 1][0], qf[nt][2 * c + 1][1]);
      }
    const int next = step + kWarps;
    if (next < end) load_k(next * kKeys);  // the fragments' registers are free: the next keys are on their way

    // s[nt][2u + e]: key index 16 step + 8u + g, row 8 nt + 2t + e
    bool raise = false;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = step * kKeys + 8 * u + g;
      const int j = key_of(i);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pp = pr[nt][e];
          const bool seen = i < n && j <= pp && (pp - j < p.window || j < p.sinks);
          float& x = s[nt][2 * u + e];
          x = seen ? x * p.scale_log2 : -INFINITY;
          raise |= x > m[nt][e] + kRescaleThreshold;
        }
    }
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
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float e0 = ex2_approx(s[nt][2 * u] - m0), e1 = ex2_approx(s[nt][2 * u + 1] - m1);
        l[nt][0] += e0;
        l[nt][1] += e1;
        // P goes to bf16 for the product (half a step, up to 2^-8 of each weight, of either sign); l keeps fp32
        pb[nt][u] = transpose_8x8(pack_bf16x2(e0, e1));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t v0[4] = {vf[0][h].x, vf[0][h].y, vf[0][h].z, vf[0][h].w};
      const uint32_t v1[4] = {vf[1][h].x, vf[1][h].y, vf[1][h].z, vf[1][h].w};
      const uint32_t v2[4] = {vf[2][h].x, vf[2][h].y, vf[2][h].z, vf[2][h].w};
      const uint32_t v3[4] = {vf[3][h].x, vf[3][h].y, vf[3][h].z, vf[3][h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = __byte_perm(v0[i], v1[i], 0x5410), a1 = __byte_perm(v0[i], v1[i], 0x7632);
        const uint32_t a2 = __byte_perm(v2[i], v3[i], 0x5410), a3 = __byte_perm(v2[i], v3[i], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816(o[4 * h + i][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
    if (next < end) load_v(next * kKeys);
  }

  // ---- join the warps: o[4h + i][nt][2f + e] is feature 64h + 8g + 2i + f of row 8 nt + 2t + e
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * t + e;
#pragma unroll
      for (int w = 4; w < 32; w *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
      if (g == 0) {
        sM[warp][r] = m[nt][e];
        sL[warp][r] = l[nt][e];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float2*>(&sO[warp][r][64 * h + 8 * g + 2 * i]) =
              make_float2(o[4 * h + i][nt][e], o[4 * h + i][nt][2 + e]);
    }
  __syncthreads();
  const int d4 = (threadIdx.x & 31) * 4;
  for (int r = warp; r < kRows; r += kWarps) {  // a warp joins a row: its partials into slot 0
    float M = sM[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sM[w][r]);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = weight(sM[w][r], M);
      const float4 v = *reinterpret_cast<const float4*>(&sO[w][r][d4]);
      L += f * sL[w][r];
      a = make_float4(a.x + f * v.x, a.y + f * v.y, a.z + f * v.z, a.w + f * v.w);
    }
    *reinterpret_cast<float4*>(&sO[0][r][d4]) = a;
    if (lane == 0) {
      cM[r] = M;
      cL[r] = L;
    }
  }
  // ---- join the cluster: row r by rank r % cluster
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int r = rank + p.cluster * warp; r < kRows; r += p.cluster * kWarps) {
    if (r0 + r >= R) break;
    float M = -INFINITY;
    for (int c = 0; c < p.cluster; ++c) M = fmaxf(M, *cluster.map_shared_rank(&cM[r], c));
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < p.cluster; ++c) {
      const float f = weight(*cluster.map_shared_rank(&cM[r], c), M);
      const float4 v = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&sO[0][r][d4], c));
      L += f * *cluster.map_shared_rank(&cL[r], c);
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

template <int NT, int kWarps>
struct Form {
  static constexpr int kSmem = sizeof(Partials<8 * NT, kWarps>);
  static const void* fn() { return reinterpret_cast<const void*>(window_split_kernel<NT, kWarps>); }

  static cudaLaunchConfig_t config(cudaLaunchAttribute* at, int cluster, long long tiles, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = static_cast<unsigned>(cluster);
    at->val.clusterDim.y = 1;
    at->val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
  }

  static DeviceOnce& allowed() {
    static DeviceOnce once;
    return once;
  }

  static int resident(const ContextKey& at, int cluster) {
    static ClusterCounts known;
    return resident_clusters(known, at, allowed(), fn(), 32 * kWarps, kSmem, cluster);
  }

  // The largest cluster with which all tiles are resident at once, every warp having a step; 0 if none.
  static int one_wave(const ContextKey& at, long long tiles, long long steps) {
    for (int c = static_cast<int>(std::min<long long>(kMaxCluster, std::max<long long>(1, steps / kWarps))); c > 0; --c)
      if (resident(at, c) >= tiles) return c;
    return 0;
  }

  static int launch(const WindowSplit& p, long long tiles, cudaStream_t stream) {
    const int rc = allow_clusters_once(allowed(), fn(), kSmem);
    if (rc != 0) return rc;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = config(&at, p.cluster, tiles, stream);
    return cudaLaunchKernelEx(&cfg, window_split_kernel<NT, kWarps>, p) == cudaSuccess ? 0 : -4;
  }
};

// How many CTAs and warps share a tile's keys. All CTAs resident at once beats
// any second wave, and more warps in flight beat fewer: of the forms with 2, 4
// and 8 warps a CTA take the one that puts most warps on the GPU in one wave
// (the smaller CTA where they tie: it fills the SMs more evenly). Four 32K-key
// windows x 40 heads, us by cluster of two-warp CTAs: 4: 388, 5: 363, 6 (a
// second wave): 459; one 2K-key window x 32 heads: two warps x 16: 12.3, four
// warps x 12: 10.8, four x 16 (a second wave): 18.
template <int NT>
int launch_rows(WindowSplit& p, long long tiles, long long steps, cudaStream_t stream) {
  const ContextKey at = current_context();
  const int c2 = Form<NT, 2>::one_wave(at, tiles, steps), c4 = Form<NT, 4>::one_wave(at, tiles, steps),
            c8 = Form<NT, 8>::one_wave(at, tiles, steps);
  if (2 * c2 >= 4 * c4 && 2 * c2 >= 8 * c8) {
    p.cluster = std::max(1, c2);
    if (c2 == 0) {
      // More tiles than fit at once. A wave costs a start of some 4 us, so one
      // CTA a tile; or, where each still has 32 steps and that hides under the
      // others' loads, the cluster (up to 8) whose last wave is fullest. us by
      // cluster 1, 2, 3, 4, 8: 2048 tiles of 129 steps 347, 324, 321, 347, 369;
      // of 17 steps 55, 61, 66, 81, 126; 4096 of 5 steps 45, 63, 80, 100, 194.
      double best = 0;
      for (int c = 1; c <= 8 && (c == 1 || c * 32 <= steps); ++c) {
        const double waves = static_cast<double>(tiles) / std::max(1, Form<NT, 2>::resident(at, c));
        const double full = waves / std::ceil(waves);
        if (full > best + 0.02) best = full, p.cluster = c;
      }
    }
    return Form<NT, 2>::launch(p, tiles, stream);
  }
  if (4 * c4 >= 8 * c8) {
    p.cluster = c4;
    return Form<NT, 4>::launch(p, tiles, stream);
  }
  p.cluster = c8;
  return Form<NT, 8>::launch(p, tiles, stream);
}

}  // namespace

// Query rows of one 16-row tile per K/V head always come here. For more, two
// estimates in us decide, fitted to forwards of 1 to 2500 query rows, 1 to 40
// heads, G from 1 to 8 and windows of 16 to 16384. This kernel: a start, each
// row tile's own, and its tensor work, whose keys feed 16 rows from registers.
// The 128-row tiles of attn_window_fwd: the visits of 256 query rows of one
// head, by one CTA or shared by a cluster. us, this kernel / tiles by one CTA /
// tiles with the cluster that the plan gives them:
//   H 32, Hkv 8, window 16384:  8 tokens 38 / 157 / 49, 32 tokens 91 / 157 / 50, 64 tokens 169 / 158 / 51
//   H 32, Hkv 32, window 1024: 32 tokens 13 / 18 / 14, 128 tokens 27 / 20 / 16
//   H 4, Hkv 4, window 4096:  256 tokens 26 / 51 / 21
//   H 4, Hkv 4, window 512:  256 tokens 10 / 17 / 15
// Of 140 other random forwards, each timed in all forms, 15 took a form that was
// more than 2% slower than the best, 4 by more than 10%, the worst by 18%. More
// row tiles than the GPU holds at once do not pay: 1024 of 256 keys take 37 and
// 512 take 20 where the tiles take 15.
bool window_split_pays(int B, int H, int Hkv, const WindowShape& w) {
  const int G = H / Hkv;
  const long long rows = static_cast<long long>(w.Sq) * G;
  if (rows <= 16) return true;
  const double row_tiles = static_cast<double>(B) * Hkv * ((rows + 15) / 16);
  if (row_tiles > 4 * kSms) return false;
  const double reach = static_cast<double>(w.window) + w.sinks + (14 + G) / G + 1;  // keys that a row tile may see
  const double keys = std::min(reach, std::max(0., std::min<double>(w.Sk, w.pos0 + 0.5 * w.Sq + 1)));
  const double split_us = 6.4 + row_tiles * (7.8e-3 + 7.7e-5 * keys) + 7.3e-4 * std::min(keys, 4096.);
  return split_us < window_tiles_us(w, B, H);
}

int launch_window_split(WindowSplit p, cudaStream_t stream) {
  if (static_cast<long long>(p.T) * (p.H / p.Hkv) > kWindowMaxRows) return -1;
  const int R = p.T * (p.H / p.Hkv);
  const int rows = R <= 8 ? 8 : 16;
  p.row_tiles = (R + rows - 1) / rows;
  // Most keys that a row tile can see, from the host's side of the sizes.
  const long long seen = std::min<long long>(p.Sk, static_cast<long long>(p.window) + p.T - 1 + p.sinks);
  const long long tiles = static_cast<long long>(p.B) * p.Hkv * p.row_tiles, steps = (seen + kKeys - 1) / kKeys;
  if (tiles > 0x7fffffffLL / kMaxCluster) return -1;
  if (tiles == 0) return 0;
  return rows == 8 ? launch_rows<1>(p, tiles, steps, stream) : launch_rows<2>(p, tiles, steps, stream);
}

}  // namespace lcb
