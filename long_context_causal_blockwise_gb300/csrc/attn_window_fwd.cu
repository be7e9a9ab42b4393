// Forward of attention with a sliding window and sinks, key/value heads shared
// by groups of query heads.
//
//   O_i = sum_j P_ij v_j over the keys j <= p that lie in the window, p - j <
//   window, or among the first `sinks`;  P = softmax(scale q.k),  LSE likewise.
//
// The tile machinery is that of the full forward: one CTA owns 256 query rows
// of a head as two 128-row tiles that ping-pong, so the tensor core works on
// one while the softmax warps work on the other; K and V stream by TMA through
// a four-slot ring; S and O live in TMEM, P goes back over S as the second
// product's A operand; the running maximum is raised lazily (by more than 2^8).
// What the window adds: a CTA streams only the key tiles that one of its rows
// can see (the sink tiles, then the window's), each query tile skips those of
// them that it does not see itself, and a tile needs the per-element mask only
// where the diagonal, the window's far edge, the last sink or the last key cuts
// it. Work is 4 * 128 flops a visible pair plus the hidden part of the cut
// tiles, at most two per query tile and edge.
//
//   warp 8      TMA producer
//   warp 9      MMA issuer (one thread), owner of the TMEM allocation
//   warps 0-3   softmax of query tile 0 (thread = query row = TMEM lane)
//   warps 4-7   softmax of query tile 1
//
// TMEM (512 columns x 128 lanes, fp32): S_0 [0,128), S_1 [128,256),
// O_0 [256,384), O_1 [384,512).
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_window.cuh"
#include "lcb_internal.h"

namespace lcb {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kD = 128;
constexpr int kStages = 4;
constexpr int kThreads = 320;
constexpr uint32_t kTileBytes = kBN * kD * 2;  // 32 KB, two 16 KB halves of 64 columns
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kSmQ = 0;
constexpr uint32_t kSmKV = 2 * kTileBytes;
constexpr uint32_t kSmBar = kSmKV + kStages * kTileBytes;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kHeadGroup = 4;              // (b, h) pairs whose query blocks interleave in the CTA order

struct Bars {
  uint64_t q_full;
  uint64_t kv_full[kStages];
  uint64_t kv_empty[kStages];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmemBytes = kSmBar + sizeof(Bars) + 1024;  // + alignment slack

struct Params {
  __nv_bfloat16* o;
  float* lse;
  long long o_rs, o_bs, l_hs, l_bs;
  int B, H, G;
  WindowShape w;
  float scale_log2;
  DevStatus st;
};

constexpr uint32_t kWhere = 5u << 24;  // kernel id of timeout reports

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }

// The visits of a CTA's two query tiles: `all` is the stream of key tiles that
// either one sees; query tile t takes part in visit i iff its own list has it.
struct Visits {
  KeyTiles all, own[2];
  int n, last[2];  // visits of the stream; the last one of each query tile (-1: none)
  __device__ __forceinline__ bool active(int t, int i) const {
    const int kt = all.tile(i);
    return i < n && (kt < own[t].ns || (kt >= own[t].lo && kt < own[t].hi));
  }
};

__device__ __forceinline__ Visits visits(const WindowShape& w, int q0) {
  Visits v;
  v.all = key_tiles(w, q0, 2 * kBM);
  v.n = v.all.count();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    v.own[t] = key_tiles(w, q0 + t * kBM, kBM);
    const int kt = v.own[t].hi > v.own[t].lo ? v.own[t].hi - 1 : v.own[t].ns - 1;  // its last key tile
    v.last[t] = kt < 0 ? -1 : (kt < v.all.ns ? kt : v.all.ns + kt - v.all.lo);
  }
  return v;
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kSmBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = static_cast<int>(warp_id());
  const int lane = static_cast<int>(lane_id());

  // (b, h) pairs go in groups of kHeadGroup, a group's CTAs latest query block
  // first with its heads interleaved: neighbours in time share K/V tiles in L2
  // (heads of one K/V head, blocks of one window), and the short first blocks
  // of the sequence end the grid.
  const int nq = (p.w.Sq + 2 * kBM - 1) / (2 * kBM);
  const int group = static_cast<int>(blockIdx.x) / (nq * kHeadGroup);
  const int g0 = group * kHeadGroup;
  const int gsz = min(kHeadGroup, p.B * p.H - g0);
  const int within = static_cast<int>(blockIdx.x) - group * nq * kHeadGroup;
  const int bh = g0 + within % gsz;
  const int b = bh / p.H, h = bh % p.H;
  const int q0 = (nq - 1 - within / gsz) * 2 * kBM;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 128);
      mbar_init(&bars->o_full[t], 1);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const Visits v = visits(p.w, q0);
    if (lane == 0 && v.n > 0) {
      const uint64_t pol = l2_policy_evict_last();
      const int xq = h * kD, xk = (h / p.G) * kD;
      const uint32_t tiles = (v.last[0] >= 0 ? 1u : 0u) + (v.last[1] >= 0 ? 1u : 0u);
      mbar_arrive_expect_tx(&bars->q_full, tiles * kTileBytes);
      for (int t = 0; t < 2; ++t) {
        if (v.last[t] < 0) continue;
        for (int half = 0; half < 2; ++half)
          tma_load_3d(smem + kSmQ + t * kTileBytes + half * kHalfBytes, &tm_q, &bars->q_full, xq + half * 64,
                      q0 + t * kBM, b);
      }
      int it = 0;
      bool ok = true;
      for (int i = 0; i < v.n && ok; ++i) {
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int slot = it % kStages;
          const uint32_t ph = static_cast<uint32_t>(it / kStages) & 1u;
          if (!mbar_wait(&bars->kv_empty[slot], ph ^ 1u, abort_flag, p.st, kWhere | (1u << 16))) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->kv_full[slot], kTileBytes);
          const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
          for (int half = 0; half < 2; ++half)
            tma_load_3d_hint(smem + kSmKV + slot * kTileBytes + half * kHalfBytes, map, &bars->kv_full[slot],
                             xk + half * 64, v.all.tile(i) * kBN, b, pol);
        }
      }
      if (!ok) {
        // Let every copy already issued land before the CTA can exit.
        drain_wait(&bars->q_full, 0, p.st.limit);
        for (int k = max(0, it - kStages); k < it; ++k)
          drain_wait(&bars->kv_full[k % kStages], static_cast<uint32_t>(k / kStages) & 1u, p.st.limit);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    const Visits v = visits(p.w, q0);
    if (lane == 0 && v.n > 0) {
      const uint32_t idesc_qk = idesc_bf16(kBM, kBN, false, false);
      const uint32_t idesc_pv = idesc_bf16(kBM, kD, false, true);
      auto issue_qk = [&](int t, int slot) {
        const uint64_t qa = sdesc_sw128(sbase + kSmQ + t * kTileBytes, 16, 1024);
        const uint64_t kb = sdesc_sw128(sbase + kSmKV + slot * kTileBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
          mma_ss(tbase + t * 128, sdesc_advance(qa, off), sdesc_advance(kb, off), idesc_qk, kk > 0);
        }
        tc_commit(&bars->s_full[t]);
      };
      auto issue_pv = [&](int t, int slot, bool acc) {
        const uint64_t vb = sdesc_sw128(sbase + kSmKV + slot * kTileBytes, kHalfBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          mma_ts(tbase + 256 + t * 128, tbase + t * 128 + kk * 8, sdesc_advance(vb, kk * 2048), idesc_pv,
                 (acc || kk > 0));
      };
      auto wait_kv = [&](int it) {
        const bool r = mbar_wait(&bars->kv_full[it % kStages], static_cast<uint32_t>(it / kStages) & 1u, abort_flag,
                                 p.st, kWhere | (3u << 16));
        tc_fence_after();
        return r;
      };
      int done[2] = {0, 0};  // products P V issued per query tile
      bool ok = mbar_wait(&bars->q_full, 0, abort_flag, p.st, kWhere | (2u << 16));
      if (ok) ok = wait_kv(0);
      if (ok) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (v.active(t, 0)) issue_qk(t, 0);
        tc_commit(&bars->kv_empty[0]);
      }
      for (int i = 0; i < v.n && ok; ++i) {
        const int itV = 2 * i + 1, itK = 2 * i + 2;
        const int sV = itV % kStages, sK = itK % kStages;
        ok = wait_kv(itV);
        if (!ok) break;
        bool k_ready = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok) continue;
          if (v.active(t, i)) {
            ok = mbar_wait(&bars->p_full[t], static_cast<uint32_t>(done[t]) & 1u, abort_flag, p.st,
                           kWhere | (4u << 16));
            if (!ok) continue;
            tc_fence_after();
            issue_pv(t, sV, done[t] > 0);
            ++done[t];
            if (i == v.last[t]) tc_commit(&bars->o_full[t]);
          }
          if (v.active(t, i + 1)) {  // S over P once the product above has read it (issue order)
            if (!k_ready) {
              ok = wait_kv(itK);
              if (!ok) continue;
              k_ready = true;
            }
            issue_qk(t, sK);
          }
        }
        if (!ok) break;
        tc_commit(&bars->kv_empty[sV]);
        if (i + 1 < v.n) tc_commit(&bars->kv_empty[sK]);
      }
      // Every MMA issued must finish before TMEM is released.
      tc_commit(&bars->mma_done);
      drain_wait(&bars->mma_done, 0, p.st.limit);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + t * 128 + lane_off;
    const uint32_t tO = tbase + 256 + t * 128 + lane_off;
    const int qi = q0 + t * kBM + row;
    const int pos = p.w.pos0 + qi;
    const int p_first = p.w.pos0 + q0 + t * kBM, p_last = p_first + kBM - 1;
    const float c = p.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const KeyTiles own = key_tiles(p.w, q0 + t * kBM, kBM);
    const int cnt = own.count();
    for (int i = 0; i < cnt; ++i) {
      ok = warp_all(mbar_wait(&bars->s_full[t], static_cast<uint32_t>(i) & 1u, abort_flag, p.st,
                              kWhere | (5u << 16)));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[128];
      tmem_ld_x128(tS, s);
      const int kbase = own.tile(i) * kBN;
      const bool whole = kbase + kBN - 1 <= p_first && kbase + kBN <= p.w.Sk &&
                         (p_last - kbase < p.w.window || kbase + kBN <= p.w.sinks);
      if (!whole) {
        // columns [from, to] are visible, and those before `sink` up to `to`
        const int to = min(pos, p.w.Sk - 1) - kbase;
        const int from = pos - p.w.window + 1 - kbase;
        const int sink = p.w.sinks - kbase;
        if (sink > 0) {
#pragma unroll
          for (int cc = 0; cc < 128; ++cc)
            if (cc > to || (cc < from && cc >= sink)) s[cc] = __float_as_uint(-INFINITY);
        } else {
#pragma unroll
          for (int cc = 0; cc < 128; ++cc)
            if (cc > to || cc < from) s[cc] = __float_as_uint(-INFINITY);
        }
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int cc = 0; cc < 128; cc += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          m4[k] = fmax3(m4[k], __uint_as_float(s[cc + 2 * k]), __uint_as_float(s[cc + 2 * k + 1]));
      const float mx = fmax3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
      const float m_new = fmaxf(m, mx * c);
      if (i == 0) {
        m = m_new;
      } else {
        const bool resc = m_new > m + kRescaleThreshold;
        if (__any_sync(0xffffffffu, resc)) {
          const float alpha = resc ? ex2_approx(m - m_new) : 1.0f;
#pragma unroll
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            tmem_ld_x32(tO + ch * 32, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st_x32(tO + ch * 32, o);
          }
          if (resc) {
            l *= alpha;
            m = m_new;
          }
        }
      }
      const float neg_m = (m == -INFINITY) ? 0.f : -m;
      // P is rounded to bf16 for the second product (half a step, 2^-9 of each weight, of either sign); l keeps fp32
      float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const int e = 64 * hf + 2 * k;
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(s[e]), __uint_as_float(s[e + 1]), c, c, neg_m, neg_m);
          const float p0 = ex2_approx(x0);
          const float p1 = ex2_approx(x1);
          if (k & 1)
            fadd2(sb0, sb1, sb0, sb1, p0, p1);
          else
            fadd2(sa0, sa1, sa0, sa1, p0, p1);
          pk[k] = pack_bf16x2(p0, p1);
        }
        tmem_st_x32(tS + 32 * hf, pk);
      }
      l += (sa0 + sb0) + (sa1 + sb1);
      tc_fence_before();
      mbar_arrive(&bars->p_full[t]);
    }
    if (ok && cnt > 0) ok = warp_all(mbar_wait(&bars->o_full[t], 0, abort_flag, p.st, kWhere | (6u << 16)));
    if (ok) {
      tc_fence_after();
      const bool valid = qi < p.w.Sq;
      const float inv_l = l == 0.f ? 0.f : 1.f / l;
      __nv_bfloat16* dst = p.o + b * p.o_bs + static_cast<long long>(qi) * p.o_rs + h * kD;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t o[32];
        if (cnt > 0) {
          tmem_ld_x32(tO + ch * 32, o);
        } else {  // no key for any row of this tile: O was never formed
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0u;
        }
        if (valid) {
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(o[k]) * inv_l, __uint_as_float(o[k + 1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(o[k + 2]) * inv_l, __uint_as_float(o[k + 3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(o[k + 4]) * inv_l, __uint_as_float(o[k + 5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(o[k + 6]) * inv_l, __uint_as_float(o[k + 7]) * inv_l);
            *reinterpret_cast<uint4*>(dst + ch * 32 + k) = w;
          }
        }
      }
      if (valid)
        p.lse[b * p.l_bs + h * p.l_hs + qi] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

}  // namespace

int launch_window_fwd(const WindowFwd& a, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  int rc;
  if ((rc = make_tma_map_bf16(&tq, a.q, a.B, a.w.Sq, a.H * kD, kBM)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tk, a.k, a.B, a.w.Sk, a.Hkv * kD, kBN)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tv, a.v, a.B, a.w.Sk, a.Hkv * kD, kBN)) != 0) return rc;
  static DeviceOnce smem_set;
  if ((rc = set_smem_limit_once(smem_set, reinterpret_cast<const void*>(attn_window_fwd_kernel), kSmemBytes)) != 0)
    return rc;
  Params p;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_rs = a.o_row_stride;
  p.o_bs = a.o_batch_stride;
  p.l_hs = a.lse_head_stride;
  p.l_bs = a.lse_batch_stride;
  p.B = a.B;
  p.H = a.H;
  p.G = a.H / a.Hkv;
  p.w = a.w;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.st = a.st;
  const long long grid = static_cast<long long>((a.w.Sq + 2 * kBM - 1) / (2 * kBM)) * a.B * a.H;
  if (grid > 0x7fffffffLL) return -1;
  attn_window_fwd_kernel<<<static_cast<unsigned>(grid), kThreads, kSmemBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
