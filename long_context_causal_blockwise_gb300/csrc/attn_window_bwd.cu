// Backward of attention with a sliding window and sinks, key/value heads
// shared by groups of query heads, in one pass.
//
// With P_ij = exp(scale q_i.k_j - LSE_i) on the visible pairs, 0 elsewhere, and
// dP_ij = dO_i.v_j, Delta_i = dO_i.O_i:
//   dS = P (dP - Delta),  dV_j = sum_i P_ij dO_i,  dK_j = scale sum_i dS_ij q_i,
//   dQ_i = scale sum_j dS_ij k_j,
// the sums over i running over all query heads that share the K/V head.
//
// The tile machinery is that of the full one-pass backward: a CTA owns 128
// keys, keeps dK and dV in TMEM, and for each (query head, query tile) pair
// forms S^T and dP^T, then dV += P^T dO, dK += dS^T Q and the partial dQ =
// dS K, added into a tiled fp32 accumulator in L2 (half of its columns by bulk
// reductions from shared memory, half by vector reductions from registers: dQ's
// summation order is not fixed). What the window adds: the pairs of a key tile
// are those whose rows reach it, for every query head of the group, so the
// shared heads' gradients are summed in the same TMEM accumulators; a pair
// needs the per-element mask only where the diagonal, the window's far edge,
// the last sink or the last key cuts it.
//
// A tile that holds sinks is seen by every later query: its list is as long as
// the sequence, and with few K/V heads its CTA would outlast the grid. Long
// lists are cut into runs, a CTA each, whose dK and dV go to fp32 partials that
// a second kernel sums in run order (so dK and dV stay deterministic).
//
// TMEM: S^T [0,128) (P^T bf16 over it), dP^T [128,256) (then the dQ partial),
// dV [256,384), dK [384,512).
//
// What bounds it: 32K tokens x 32 heads, window 4096, take 4.45 ms: 4330 clocks
// a pair of which the products need 2560, at 1.96 GHz under the 1.4 kW cap. By
// time stamps the compute warps are busy or in short waits throughout (dS 780
// clocks, P 830, the dQ export 1040 to 1380, waits 1400). None of these moved
// it: two groups of eight warps on alternate pairs (8% slower), the dQ export
// in warps of its own (4% slower), -LSE added by the tensor core as one more
// K step (no change), the last steps of dK after the next dP^T (13% slower: the
// one dS buffer then waits for them), Q and dO freed and loaded by halves (no
// change). Waits without a function call, which had cost spills: 6.62 -> 6.21
// ms with the forward.
//
// Shared memory: K, V, a two-slot Q ring with the row statistics of its tile,
// one dO slot, dS^T, two 16 KB staging blocks for dQ.
// Warps 0-15 compute, 16 TMA producer, 17 MMA issuer, 18 dQ reducer.
#include <algorithm>

#include "attn_window.cuh"
#include "lcb_attn.h"
#include "lcb_internal.h"
#include "mma_warp.cuh"

namespace lcb {
namespace {

constexpr int kT = 128;  // rows of every tile
constexpr int kD = 128;
constexpr int kCompute = 512;  // compute threads: warps 0-15
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
constexpr int kReduceWarp = 18;
constexpr int kThreads = 608;
constexpr uint32_t kTileBytes = kT * kD * 2;   // 32 KB: two 16 KB boxes of 128 rows x 64 columns
constexpr uint32_t kColHalf = kTileBytes / 2;  // column-half stride of a tile
constexpr uint32_t kDqBlock = 128 * 32 * 4;    // one staged dQ block: 128 rows x 32 columns fp32
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Loads one 128-row tile (two 64-column boxes) of `map` at row `row`.
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int x0, int row, int b,
                                          uint64_t pol) {
  tma_load_3d_hint(dst, map, bar, x0, row, b, pol);
  tma_load_3d_hint(dst + kColHalf, map, bar, x0 + 64, row, b, pol);
}

// Writes 32 bf16 values (16 packed words) as columns [32q, 32q+32) of row `r`
// of a 128 x 128 K-major tile with 128-byte swizzle (the layout TMA produces).
__device__ __forceinline__ void st_tile_quarter_row(uint8_t* tile, int r, int q, const uint32_t (&w)[16]) {
  uint8_t* rowp = tile + (q >> 1) * kColHalf + r * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int ch = 4 * (q & 1) + c;
    *reinterpret_cast<uint4*>(rowp + ((ch ^ (r & 7)) << 4)) =
        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

// Stores 32 columns of a gradient row, fp32 accumulator values, as bf16 or as they are.
__device__ __forceinline__ void store_row(void* base, long long off, const uint32_t (&a)[32], bool f32) {
  if (f32) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i] = make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off);
    auto pair = [&](int i) { return pack_bf16x2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])); };
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(pair(8 * i), pair(8 * i + 2), pair(8 * i + 4), pair(8 * i + 6));
  }
}

__device__ __forceinline__ void bulk_reduce_add_f32(float* gdst, uint32_t ssrc, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(gdst), "r"(ssrc),
               "r"(bytes)
               : "memory");
}
// Adds four floats at gaddr (16-byte aligned) in L2, fire and forget.
__device__ __forceinline__ void red_add_v4(float* gaddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(gaddr), "f"(__uint_as_float(a)),
               "f"(__uint_as_float(b)), "f"(__uint_as_float(c)), "f"(__uint_as_float(d))
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

struct WinBars {
  uint64_t fixed_full;             // K and V are in place
  uint64_t q_full[2], q_empty[2];  // Q ring (and its statistics), by the pair's parity
  uint64_t do_full, do_empty;      // the dO slot
  uint64_t s_full, dp_full;        // S^T, dP^T computed
  uint64_t p_full;                 // P^T in TMEM
  uint64_t ds_full;                // dS^T in shared memory, dP^T in registers
  uint64_t ds_free;                // the products that read dS^T are done
  uint64_t dq_full, dq_free;       // the dQ partial computed; loaded by every compute thread
  uint64_t stg_full[2], stg_free[2];  // warpgroup x's (x = 0, 1) dQ block staged; read by the reducer
  uint64_t acc_full, mma_done;
  uint32_t tmem_base;
  int abort;
};

constexpr uint32_t kStatBytes = 2 * kT * 4;  // a tile's row statistics: -LSE log2 e, then -scale Delta
constexpr uint32_t kWinSmK = 0;
constexpr uint32_t kWinSmV = kTileBytes;
constexpr uint32_t kWinSmQ = 2 * kTileBytes;
constexpr uint32_t kWinSmDo = kWinSmQ + 2 * kTileBytes;
constexpr uint32_t kWinSmDs = kWinSmDo + kTileBytes;
constexpr uint32_t kWinSmStg = kWinSmDs + kTileBytes;
constexpr uint32_t kWinSmStat = kWinSmStg + 2 * kDqBlock;
constexpr uint32_t kWinSmBar = kWinSmStat + 2 * kStatBytes;
constexpr uint32_t kWinSmem = kWinSmBar + sizeof(WinBars) + 512;  // + what aligning to 1024 may take
static_assert(kWinSmem <= 232448, "shared memory of one CTA");

struct WinParams {
  const __nv_bfloat16* o;
  const __nv_bfloat16* dO;
  long long o_rs, o_bs;
  const float* lse;
  long long l_hs, l_bs;
  float* stats;  // [B, H, 2, tiles * 128]: the two row statistics, padded to whole tiles
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  long long dq_rs, dq_bs, g_rs, g_bs;
  float* dq_acc;  // [B, H, tiles] tiles of 128 x 128
  float* partial;
  int B, H, Hkv, q_tiles;
  WindowShape w;
  WindowBwdPlan plan;
  float scale, scale_log2;
  DevStatus st;
};

// Before the pass: the row statistics, and zeros for the dQ accumulator. One
// warp a token row (rows past the last fill their tile: LSE = -inf gives P = 0)
// over all heads, half a warp a head's dO.O (O as the forward rounded it, the
// sum in fp32), eight heads' loads in flight.
// Bound by HBM: 512 bytes read and 520 written per row and head.
__global__ void __launch_bounds__(256) window_bwd_prep_kernel(const __grid_constant__ WinParams p) {
  const int rows = p.q_tiles * kT;
  const int ln = threadIdx.x & 31, half = ln >> 4;
  const long long n = static_cast<long long>(p.B) * rows, step = static_cast<long long>(gridDim.x) * 8;
  for (long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); w < n; w += step) {
    const int b = static_cast<int>(w / rows), s = static_cast<int>(w % rows);
    const long long row = b * p.o_bs + static_cast<long long>(s) * p.o_rs + (ln & 15) * 8;
    const bool in = s < p.w.Sq;
    for (int h0 = 0; h0 < p.H; h0 += 8) {
      uint4 x[4], y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int h = h0 + 2 * u + half;
        x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
        if (in && h < p.H) {
          x[u] = __ldg(reinterpret_cast<const uint4*>(p.o + row + h * kD));
          y[u] = __ldg(reinterpret_cast<const uint4*>(p.dO + row + h * kD));
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int h = h0 + u;
        if (h < p.H)
          reinterpret_cast<float4*>(p.dq_acc + (static_cast<long long>(b) * p.H + h) * rows * kD +
                                    static_cast<long long>(s) * kD)[ln] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t xs[4] = {x[u].x, x[u].y, x[u].z, x[u].w}, ys[4] = {y[u].x, y[u].y, y[u].z, y[u].w};
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d += bf16lo_to_f32(xs[e]) * bf16lo_to_f32(ys[e]) + bf16hi_to_f32(xs[e]) * bf16hi_to_f32(ys[e]);
#pragma unroll
        for (int k = 8; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
        const int h = h0 + 2 * u + half;
        if ((ln & 15) == 0 && h < p.H) {
          float* st = p.stats + (static_cast<long long>(b) * p.H + h) * 2 * rows + s;
          const float l = in ? p.lse[b * p.l_bs + h * p.l_hs + s] : -INFINITY;
          // an empty row (LSE = -inf) must give P = 0
          st[0] = l == -INFINITY ? -INFINITY : -l * kLog2e;
          st[rows] = -p.scale * d;
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_window_bwd_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                           const __grid_constant__ WinParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t gap = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  if (gap > 512u) {  // dynamic shared memory starts on 1024 bytes; were it not to, the tiles would not fit
    if (threadIdx.x == 0) atomicOr(p.st.words, DEV_TIMEOUT);
    return;
  }
  uint8_t* smem = smem_raw + gap;
  const uint32_t sbase = smem_u32(smem);
  WinBars* bars = reinterpret_cast<WinBars*>(smem + kWinSmBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = static_cast<int>(uniform(warp_id()));
  const int lane = static_cast<int>(lane_id());
  constexpr uint32_t kWhere = 6u << 24;

  // Work item: the sink tiles' runs come first (the longest lists), then the
  // other key tiles, head by head, so that the CTAs running together read the
  // query tiles and add into the dQ tiles of one stretch of a few heads.
  const bool sink = static_cast<long long>(blockIdx.x) < p.plan.sink_ctas;
  const int local = static_cast<int>(blockIdx.x) - (sink ? 0 : static_cast<int>(p.plan.sink_ctas));
  const int segs = sink ? p.plan.sink_segs : p.plan.segs;
  const int tiles = sink ? p.plan.sink_tiles : p.plan.key_tiles - p.plan.sink_tiles;
  const int seg = local % segs;
  const int kt = (local / segs) % tiles + (sink ? 0 : p.plan.sink_tiles);
  const int bh = local / segs / tiles;
  const int b = bh / p.Hkv, hk = bh % p.Hkv;
  const int G = p.H / p.Hkv;
  const QueryTiles qt = query_tiles(p.w, kt);
  const int per = qt.hi - qt.lo;
  const int all = G * per;
  const int run = (all + segs - 1) / segs;
  const int s0 = min(all, seg * run);
  const int n = min(all, s0 + run) - s0;  // pairs of this CTA: s0 .. s0 + n - 1 of the list, head-major
  auto head_of = [&](int i) { return hk * G + (s0 + i) / per; };
  auto tile_of = [&](int i) { return qt.lo + (s0 + i) % per; };

  if (threadIdx.x == 0) {
    mbar_init(&bars->fixed_full, 1);
    mbar_init(&bars->do_full, 1);
    mbar_init(&bars->do_empty, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_full, kCompute);
    mbar_init(&bars->ds_full, kCompute);
    mbar_init(&bars->ds_free, 1);
    mbar_init(&bars->dq_full, 1);
    mbar_init(&bars->dq_free, kCompute);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->q_full[x], 1);
      mbar_init(&bars->q_empty[x], 1);
      mbar_init(&bars->stg_full[x], 128);
      mbar_init(&bars->stg_free[x], 1);
    }
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  const uint32_t tS = tbase, tDP = tbase + 128, tDV = tbase + 256, tDK = tbase + 384;
  const uint32_t tDQ = tDP;

  if (warp == kProducerWarp) {
    if (lane == 0 && n > 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_do);
      const uint64_t pol = l2_policy_evict_last();
      mbar_arrive_expect_tx(&bars->fixed_full, 2 * kTileBytes);
      load_tile(smem + kWinSmK, &tm_k, &bars->fixed_full, hk * kD, kt * kT, b, pol);
      load_tile(smem + kWinSmV, &tm_v, &bars->fixed_full, hk * kD, kt * kT, b, pol);
      int nq = 0, nd = 0;  // Q and dO tiles under way
      for (int i = 0; i < n; ++i) {
        const int s = i & 1, h = head_of(i), t = tile_of(i);
        if (!mbar_wait_inline(&bars->q_empty[s], ((i >> 1) & 1) ^ 1, abort_flag, p.st, kWhere | (1u << 16))) break;
        mbar_arrive_expect_tx(&bars->q_full[s], kTileBytes + kStatBytes);
        load_tile(smem + kWinSmQ + s * kTileBytes, &tm_q, &bars->q_full[s], h * kD, t * kT, b, pol);
        const float* st =
            p.stats + (static_cast<long long>(b) * p.H + h) * 2 * p.q_tiles * kT + static_cast<long long>(t) * kT;
        bulk_load(smem + kWinSmStat + s * kStatBytes, st, kT * 4, &bars->q_full[s]);
        bulk_load(smem + kWinSmStat + s * kStatBytes + kT * 4, st + static_cast<long long>(p.q_tiles) * kT, kT * 4,
                  &bars->q_full[s]);
        ++nq;
        if (!mbar_wait_inline(&bars->do_empty, (i & 1) ^ 1, abort_flag, p.st, kWhere | (11u << 16))) break;
        mbar_arrive_expect_tx(&bars->do_full, kTileBytes);
        load_tile(smem + kWinSmDo, &tm_do, &bars->do_full, h * kD, t * kT, b, pol);
        ++nd;
      }
      if (nd < n) {
        // Every copy already issued lands before the CTA can exit.
        drain_wait(&bars->fixed_full, 0, p.st.limit);
        for (int i = max(0, nq - 2); i < nq; ++i) drain_wait(&bars->q_full[i & 1], (i >> 1) & 1, p.st.limit);
        if (nd > 0) drain_wait(&bars->do_full, (nd - 1) & 1, p.st.limit);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // All lanes walk the loop, one elected lane issues.
    if (n > 0) {
      const uint32_t one = elect_one();
      const uint32_t tm = uniform(tbase);
      const uint32_t uS = tm, uDP = tm + 128, uDV = tm + 256, uDK = tm + 384, uDQ = uDP;
      const uint32_t id_s = idesc_bf16(kT, kT, false, false);  // scores: both operands K-major
      const uint32_t id_g = idesc_bf16(kT, kD, false, true);   // dK, dV: B MN-major
      const uint32_t id_q = idesc_bf16(kT, kD, true, true);    // dQ: A (dS) and B (K) MN-major
      // operands as read K-major (rows) and MN-major (columns)
      const uint64_t k_rows = sdesc_sw128(sbase + kWinSmK, 16, 1024),
                     k_cols = sdesc_sw128(sbase + kWinSmK, kColHalf, 1024);
      const uint64_t v_rows = sdesc_sw128(sbase + kWinSmV, 16, 1024);
      const uint64_t q_rows = sdesc_sw128(sbase + kWinSmQ, 16, 1024),
                     q_cols = sdesc_sw128(sbase + kWinSmQ, kColHalf, 1024);
      const uint64_t do_rows = sdesc_sw128(sbase + kWinSmDo, 16, 1024),
                     do_cols = sdesc_sw128(sbase + kWinSmDo, kColHalf, 1024);
      const uint64_t ds_rows = sdesc_sw128(sbase + kWinSmDs, 16, 1024),
                     ds_cols = sdesc_sw128(sbase + kWinSmDs, kColHalf, 1024);
      auto slot = [&](int i) { return static_cast<uint32_t>(i & 1) * kTileBytes; };
      auto scores = [&](uint32_t d, uint64_t da, uint64_t db) {  // D = A B^T, both K-major
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * kColHalf + (kk & 3) * 32;
          mma_ss_if(d, sdesc_advance(da, off), sdesc_advance(db, off), id_s, kk > 0, one);
        }
      };
      auto wait = [&](uint64_t* bar, int ph, uint32_t id) {
        const bool r = mbar_wait_warp(bar, static_cast<uint32_t>(ph) & 1u, abort_flag, p.st, kWhere | (id << 16));
        tc_fence_after();
        return r;
      };
      bool ok = wait(&bars->fixed_full, 0, 2u) && wait(&bars->q_full[0], 0, 3u);
      if (ok) {
        scores(uS, k_rows, q_rows);  // S^T(0) = K Q_0^T
        tc_commit_if(&bars->s_full, one);
        ok = wait(&bars->do_full, 0, 12u);
      }
      if (ok) {
        scores(uDP, v_rows, do_rows);  // dP^T(0) = V dO_0^T
        tc_commit_if(&bars->dp_full, one);
      }
      for (int i = 0; i < n && ok; ++i) {
        const int x = i & 1;  // its Q slot
        const uint32_t acc = i > 0 ? 1u : 0u;
        ok = wait(&bars->p_full, i, 4u);
        if (!ok) break;
        // dV += P^T(i) dO_i; P^T K-step kk (queries 16kk..16kk+15) sits at columns 32(kk/2) + 8(kk%2)
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_if(uDV, uS + 32 * (kk >> 1) + 8 * (kk & 1), sdesc_advance(do_cols, kk * 2048), id_g,
                    kk > 0 ? 1u : acc, one);
        tc_commit_if(&bars->do_empty, one);  // the dO slot may take dO(i+1)
        if (i + 1 < n) {
          ok = wait(&bars->q_full[x ^ 1], (i + 1) >> 1, 3u);
          if (!ok) break;
          scores(uS, k_rows, sdesc_advance(q_rows, slot(i + 1)));  // S^T(i+1), after dV read P^T(i)
          tc_commit_if(&bars->s_full, one);
        }
        // dS^T(i) is in shared memory, and dP^T(i) in registers
        ok = wait(&bars->ds_full, i, 13u);
        if (!ok) break;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // dQ(i) = dS(i) K
          mma_ss_if(uDQ, sdesc_advance(ds_cols, kk * 2048), sdesc_advance(k_cols, kk * 2048), id_q, kk > 0, one);
        tc_commit_if(&bars->dq_full, one);
        const uint64_t qi = sdesc_advance(q_cols, slot(i));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // dK += dS^T(i) Q_i
          mma_ss_if(uDK, sdesc_advance(ds_rows, (kk >> 2) * kColHalf + (kk & 3) * 32), sdesc_advance(qi, kk * 2048),
                    id_g, kk > 0 ? 1u : acc, one);
        tc_commit_if(&bars->ds_free, one);
        tc_commit_if(&bars->q_empty[x], one);
        if (i + 1 < n) {
          ok = wait(&bars->do_full, i + 1, 12u) && wait(&bars->dq_free, i, 8u);
          if (!ok) break;
          scores(uDP, v_rows, do_rows);  // dP^T(i+1), over the read dQ(i)
          tc_commit_if(&bars->dp_full, one);
        }
      }
      if (ok) tc_commit_if(&bars->acc_full, one);
      tc_commit_if(&bars->mma_done, one);
      drain_wait(&bars->mma_done, 0, p.st.limit);
    }
    __syncwarp();
  } else if (warp == kReduceWarp) {
    // Adds the two staged 16 KB dQ blocks of each pair (columns 0-63) into the
    // accumulator and frees each slot once read.
    if (lane == 0 && n > 0) {
      for (int i = 0; i < n; ++i) {
        const uint32_t ph = static_cast<uint32_t>(i) & 1u;
        float* tile = p.dq_acc + ((static_cast<long long>(b) * p.H + head_of(i)) * p.q_tiles + tile_of(i)) * (kT * kD);
        if (!mbar_wait_inline(&bars->stg_full[0], ph, abort_flag, p.st, kWhere | (14u << 16))) break;
        bulk_reduce_add_f32(tile, sbase + kWinSmStg, kDqBlock);
        bulk_commit();
        if (!mbar_wait_inline(&bars->stg_full[1], ph, abort_flag, p.st, kWhere | (14u << 16))) break;
        bulk_reduce_add_f32(tile + kDqBlock / 4, sbase + kWinSmStg + kDqBlock, kDqBlock);
        bulk_commit();
        bulk_wait_read<1>();
        mbar_arrive(&bars->stg_free[0]);
        bulk_wait_read<0>();
        mbar_arrive(&bars->stg_free[1]);
      }
      bulk_wait_all();  // every reduction issued has completed
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- compute
    const int x = warp >> 2;            // this warpgroup's query columns [32x, 32x + 32)
    const int row = threadIdx.x & 127;  // key row of S^T/dP^T/dV/dK, query row of dQ: the TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint8_t* ds_tile = smem + kWinSmDs;
    uint8_t* stg_row = smem + kWinSmStg + (x & 1) * kDqBlock + row * 128;  // used by warpgroups 0 and 1
    const int j0 = kt * kT, j = j0 + row;
    const bool key_ok = j < p.w.Sk;  // a zero-filled row past the last key: P must be 0
    const float c = p.scale_log2;
    // The statistics of this warpgroup's queries, read as broadcasts from pair i's ring slot.
    auto stats = [&](int i) {
      return reinterpret_cast<const float*>(smem + kWinSmStat + (i & 1) * kStatBytes) + 32 * x;
    };
    bool ok = true;
    // Step s runs phase 2 of pair s-1, phase 1 of pair s, then phase 3 of pair
    // s-1: P^T(s) is computed while the tensor pipe runs dQ(s-1) and dK(s-1).
    float pv[32];  // P^T of the pair between its phases 1 and 2
    const float scl = p.scale;
    for (int s = 0; s <= n && ok; ++s) {
      if (s > 0) {
        // Phase 2: dS'^T = scale P^T (dP^T - Delta), rounded to bf16 (half a step, up to 2^-8 of each value, of
        // either sign) into shared memory for dK and dQ, which come out of the products scaled.
        const int i = s - 1;
        const uint32_t ph = static_cast<uint32_t>(i) & 1u;
        ok = mbar_wait_warp(&bars->dp_full, ph, abort_flag, p.st, kWhere | (6u << 16));
        if (!ok) break;
        tc_fence_after();
        const float* sds = stats(i) + kT;
        uint32_t dk[16];
        {
          uint32_t dp[32];
          tmem_ld_x32(tDP + lane_off + 32 * x, dp);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 d = *reinterpret_cast<const float4*>(sds + e);
            float t0, t1, u0, u1;
            ffma2(t0, t1, __uint_as_float(dp[e]), __uint_as_float(dp[e + 1]), scl, scl, d.x, d.y);
            fmul2(u0, u1, pv[e], pv[e + 1], t0, t1);
            dk[e >> 1] = pack_bf16x2(u0, u1);
            ffma2(t0, t1, __uint_as_float(dp[e + 2]), __uint_as_float(dp[e + 3]), scl, scl, d.z, d.w);
            fmul2(u0, u1, pv[e + 2], pv[e + 3], t0, t1);
            dk[(e >> 1) + 1] = pack_bf16x2(u0, u1);
          }
        }
        if (i > 0) {
          ok = mbar_wait_warp(&bars->ds_free, ph ^ 1u, abort_flag, p.st, kWhere | (9u << 16));
          if (!ok) break;
        }
        st_tile_quarter_row(ds_tile, row, x, dk);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&bars->ds_full);  // also: dP^T(i) is in registers, its columns may take dQ(i)
      }
      if (s < n) {
        // Phase 1: P^T(s), into this warpgroup's own S^T columns (already read by it).
        const int p0 = p.w.pos0 + tile_of(s) * kT;  // position of the pair's first query
        ok = mbar_wait_warp(&bars->s_full, static_cast<uint32_t>(s) & 1u, abort_flag, p.st, kWhere | (5u << 16)) &&
             mbar_wait_warp(&bars->q_full[s & 1], static_cast<uint32_t>(s >> 1) & 1u, abort_flag, p.st,
                            kWhere | (3u << 16));
        if (!ok) break;
        tc_fence_after();
        const float* l2s = stats(s);
        const bool whole = j0 + kT - 1 <= p0 && j0 + kT <= p.w.Sk &&
                           (p0 + kT - 1 - j0 < p.w.window || j0 + kT <= p.w.sinks);
        {
          uint32_t sv[32];
          tmem_ld_x32(tS + lane_off + 32 * x, sv);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 m = *reinterpret_cast<const float4*>(l2s + e);
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]), c, c, m.x, m.y);
            pv[e] = ex2_approx(x0);
            pv[e + 1] = ex2_approx(x1);
            ffma2(x0, x1, __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]), c, c, m.z, m.w);
            pv[e + 2] = ex2_approx(x0);
            pv[e + 3] = ex2_approx(x1);
          }
          if (!whole) {
            // queries 32x + e with e in [from, to] of this tile see key j
            const int at = p0 + 32 * x;
            const int from = j - at;
            const int to = !key_ok ? -1 : (j < p.w.sinks ? 31 : j + (p.w.window - 1) - at);
            const uint32_t see = low_bits(to + 1) & ~low_bits(from);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) pv[e] = 0.f;
          }
        }
        {
          // to bf16 for dV (half a step, up to 2^-8 of each weight, of either sign); dS takes the fp32 values
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) pk[e >> 1] = pack_bf16x2(pv[e], pv[e + 1]);
          tmem_st_x16_nowait(tS + lane_off + 32 * x, pk);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&bars->p_full);  // dV(s) and S^T(s+1) may go
      }
      if (s > 0) {
        // Phase 3: row `row` of dQ(i) (TMEM lane = query row), columns [32x, 32x + 32), added into the accumulator.
        const int i = s - 1;
        const uint32_t ph = static_cast<uint32_t>(i) & 1u;
        ok = mbar_wait_warp(&bars->dq_full, ph, abort_flag, p.st, kWhere | (7u << 16));
        if (!ok) break;
        tc_fence_after();
        uint32_t g[32];
        tmem_ld_x32(tDQ + lane_off + 32 * x, g);
        tc_fence_before();
        mbar_arrive(&bars->dq_free);
        if (x < 2) {
          if (i > 0)
            ok = mbar_wait_warp(&bars->stg_free[x], ph ^ 1u, abort_flag, p.st, kWhere | (15u << 16));
          if (!ok) break;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            *reinterpret_cast<uint4*>(stg_row + ((ch ^ (row & 7)) << 4)) =
                make_uint4(g[4 * ch], g[4 * ch + 1], g[4 * ch + 2], g[4 * ch + 3]);
          fence_proxy_async_smem();
          mbar_arrive(&bars->stg_full[x]);
        } else {
          float* tile =
              p.dq_acc + ((static_cast<long long>(b) * p.H + head_of(i)) * p.q_tiles + tile_of(i)) * (kT * kD);
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            red_add_v4(tile + 8192 + ((8 * (x - 2) + ch) * 128 + row) * 4, g[4 * ch], g[4 * ch + 1], g[4 * ch + 2],
                       g[4 * ch + 3]);
        }
      }
    }
    // Epilogue: a quarter of the warps each for dV columns [0,64), [64,128), and dK's; bf16 rows, or this run's partial.
    const int quarter = warp >> 2;
    const bool parts = segs > 1;
    const bool valid = parts || key_ok;
    const int half = quarter & 1;
    const long long at_slot = static_cast<long long>(local) + (!sink && p.plan.split(true) ? p.plan.sink_ctas : 0);
    void* gdst;
    long long off;
    if (parts) {
      gdst = p.partial;
      off = (at_slot * 2 + (quarter < 2 ? 1 : 0)) * (kT * kD) + row * kD + 64 * half;
    } else {
      gdst = quarter < 2 ? p.dv : p.dk;
      off = b * p.g_bs + static_cast<long long>(j) * p.g_rs + hk * kD + 64 * half;
    }
    const uint32_t tacc = (quarter < 2 ? tDV : tDK) + lane_off + 64 * half;
    if (n > 0 && ok) ok = mbar_wait_warp(&bars->acc_full, 0, abort_flag, p.st, kWhere | (10u << 16));
    if (ok) {
      tc_fence_after();
#pragma unroll 1
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t a[32];
        if (n > 0) {
          tmem_ld_x32(tacc + ch * 32, a);
        } else {  // no query sees these keys
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = 0u;
        }
        if (valid) store_row(gdst, off + ch * 32, a, parts);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// After the pass: dQ from its tiled fp32 accumulator to bf16 rows (the first
// `dq_blocks` CTAs, 16 rows of a tile each), and dK, dV of the split key tiles,
// their runs' fp32 partials summed in run order and rounded once (16 rows of
// one tile's dK or dV a CTA). A thread has eight columns of a row.
__global__ void __launch_bounds__(256) window_bwd_finish_kernel(const __grid_constant__ WinParams p, int dq_blocks,
                                                                int sink_blocks) {
  const int r16 = static_cast<int>(threadIdx.x >> 4), k16 = threadIdx.x & 15;
  int id = static_cast<int>(blockIdx.x);
  float4 a, c;
  __nv_bfloat16* dst;
  if (id < dq_blocks) {
    const int tile = id >> 3, row = (id & 7) * 16 + r16;
    const int t = tile % p.q_tiles, bh = tile / p.q_tiles;
    const int s = t * kT + row;
    if (s >= p.w.Sq) return;
    const float* tl = p.dq_acc + static_cast<long long>(tile) * (kT * kD);
    if (k16 < 8) {  // columns 0-63: 32-column blocks, chunks swizzled by row
      const float* src = tl + (k16 >> 2) * 4096 + row * 32;
      const int ch = (k16 & 3) * 2;
      a = __ldg(reinterpret_cast<const float4*>(src + ((ch ^ (row & 7)) << 2)));
      c = __ldg(reinterpret_cast<const float4*>(src + (((ch + 1) ^ (row & 7)) << 2)));
    } else {  // columns 64-127: chunk-major
      const float* src = tl + 8192 + ((2 * k16 - 16) * 128 + row) * 4;
      a = __ldg(reinterpret_cast<const float4*>(src));
      c = __ldg(reinterpret_cast<const float4*>(src + 512));
    }
    dst = p.dq + bh / p.H * p.dq_bs + static_cast<long long>(s) * p.dq_rs + (bh % p.H) * kD + k16 * 8;
  } else {
    id -= dq_blocks;
    const bool sink = id < sink_blocks;
    if (!sink) id -= sink_blocks;
    const int part = id % 16;  // 8 groups of rows, dK then dV
    id /= 16;
    const int tiles = sink ? p.plan.sink_tiles : p.plan.key_tiles - p.plan.sink_tiles;
    const int segs = sink ? p.plan.sink_segs : p.plan.segs;
    const int kt = id % tiles + (sink ? 0 : p.plan.sink_tiles), bh = id / tiles;
    const int row = (part & 7) * 16 + r16;
    const int j = kt * kT + row;
    if (j >= p.w.Sk) return;
    const long long slot = static_cast<long long>(id) * segs + (!sink && p.plan.split(true) ? p.plan.sink_ctas : 0);
    const float* src = p.partial + (slot * 2 + (part >> 3)) * (kT * kD) + row * kD + k16 * 8;
    a = c = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < segs; ++s, src += 2 * kT * kD) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(src)), v = __ldg(reinterpret_cast<const float4*>(src) + 1);
      a = make_float4(a.x + u.x, a.y + u.y, a.z + u.z, a.w + u.w);
      c = make_float4(c.x + v.x, c.y + v.y, c.z + v.z, c.w + v.w);
    }
    dst = ((part >> 3) ? p.dv : p.dk) + bh / p.Hkv * p.g_bs + static_cast<long long>(j) * p.g_rs + (bh % p.Hkv) * kD +
          k16 * 8;
  }
  *reinterpret_cast<uint4*>(dst) =
      make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(c.x, c.y), pack_bf16x2(c.z, c.w));
}

}  // namespace

WindowBwdPlan plan_window_bwd(const WindowShape& w, int B, int H, int Hkv) {
  WindowBwdPlan pl = {};
  const long long heads = static_cast<long long>(B) * Hkv, G = H / Hkv;
  pl.key_tiles = (w.Sk + kT - 1) / kT;
  pl.sink_tiles = std::min(pl.key_tiles, (w.sinks + kT - 1) / kT);
  long long pairs = 0, longest = 0, longest_sink = 0;
  for (int kt = 0; kt < pl.key_tiles; ++kt) {
    const QueryTiles q = query_tiles(w, kt);
    const long long n = G * (q.hi - q.lo);
    pairs += n * heads;
    (kt < pl.sink_tiles ? longest_sink : longest) = std::max(kt < pl.sink_tiles ? longest_sink : longest, n);
  }
  // A run is long enough for its fixed cost (loading K and V, writing dK and
  // dV: about two pairs' time) and short enough that about three of them could
  // follow one another on every SM.
  const long long run = std::max<long long>(8, (pairs + 152 * 3 - 1) / (152 * 3));
  pl.segs = static_cast<int>(std::max<long long>(1, (longest + run - 1) / run));
  pl.sink_segs = static_cast<int>(std::max<long long>(1, (longest_sink + run - 1) / run));
  pl.sink_ctas = heads * pl.sink_tiles * pl.sink_segs;
  const long long rest = heads * (pl.key_tiles - pl.sink_tiles) * pl.segs;
  pl.ctas = pl.sink_ctas + rest;
  pl.slots = (pl.sink_segs > 1 ? pl.sink_ctas : 0) + (pl.segs > 1 ? rest : 0);
  return pl;
}

int launch_window_bwd(const WindowBwd& a, cudaStream_t stream) {
  CUtensorMap tk, tv, tq, tdo;
  int rc;
  if ((rc = make_tma_map_bf16(&tk, a.k, a.B, a.w.Sk, a.Hkv * kD, kT)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tv, a.v, a.B, a.w.Sk, a.Hkv * kD, kT)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tq, a.q, a.B, a.w.Sq, a.H * kD, kT)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tdo, a.dO, a.B, a.w.Sq, a.H * kD, kT)) != 0) return rc;
  static DeviceOnce smem_set;
  if ((rc = set_smem_limit_once(smem_set, reinterpret_cast<const void*>(attn_window_bwd_kernel), kWinSmem)) != 0)
    return rc;
  WinParams p;
  p.o = static_cast<const __nv_bfloat16*>(a.o.ptr);
  p.dO = static_cast<const __nv_bfloat16*>(a.dO.ptr);
  p.o_rs = a.o.row_stride;
  p.o_bs = a.o.batch_stride;
  p.lse = a.lse;
  p.l_hs = a.lse_head_stride;
  p.l_bs = a.lse_batch_stride;
  p.dq = static_cast<__nv_bfloat16*>(a.dq);
  p.dk = static_cast<__nv_bfloat16*>(a.dk);
  p.dv = static_cast<__nv_bfloat16*>(a.dv);
  p.dq_rs = a.dq_row_stride;
  p.dq_bs = a.dq_batch_stride;
  p.g_rs = a.dkv_row_stride;
  p.g_bs = a.dkv_batch_stride;
  p.q_tiles = (a.w.Sq + kT - 1) / kT;
  const long long q_tiles = static_cast<long long>(a.B) * a.H * p.q_tiles;
  p.stats = a.workspace;
  p.dq_acc = p.stats + q_tiles * 2 * kT;
  p.partial = p.dq_acc + q_tiles * kT * kD;
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.w = a.w;
  p.plan = plan_window_bwd(a.w, a.B, a.H, a.Hkv);
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  p.st = a.st;
  const long long heads = static_cast<long long>(a.B) * a.Hkv;
  const long long dq_blocks = q_tiles * 8;
  const long long sink_blocks = p.plan.split(true) ? heads * p.plan.sink_tiles * 16 : 0;
  const long long rest_blocks = p.plan.split(false) ? heads * (p.plan.key_tiles - p.plan.sink_tiles) * 16 : 0;
  if (p.plan.ctas > 0x7fffffffLL || dq_blocks + sink_blocks + rest_blocks > 0x7fffffffLL) return -1;
  const long long rows = static_cast<long long>(a.B) * p.q_tiles * kT;
  window_bwd_prep_kernel<<<static_cast<unsigned>(std::min<long long>(rows / 8, 152LL * 16)), 256, 0, stream>>>(p);
  attn_window_bwd_kernel<<<static_cast<unsigned>(p.plan.ctas), kThreads, kWinSmem, stream>>>(tk, tv, tq, tdo, p);
  window_bwd_finish_kernel<<<static_cast<unsigned>(dq_blocks + sink_blocks + rest_blocks), 256, 0, stream>>>(
      p, static_cast<int>(dq_blocks), static_cast<int>(sink_blocks));
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
