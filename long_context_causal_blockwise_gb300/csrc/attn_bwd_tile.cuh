// Tile-level building blocks of the backward kernels: their barriers, tile
// loads, the 128 x 128 x 128 products, the swizzled dS store, gradient stores
// and the one-pass kernels' shared-memory layout and dQ reductions.
//
// Every product is M = 128 x N = 128, issued as K = 16 steps. Warps 0-15 of a
// backward kernel are its four compute warpgroups, warp 16 the TMA producer,
// warp 17 the MMA issuer and TMEM owner.
#pragma once

#include <cuda_bf16.h>

#include "lcb_attn.h"
#include "lcb_internal.h"

namespace lcb {
namespace {

constexpr int kT = 128;  // rows of every tile
constexpr int kD = 128;
constexpr int kThreads = 576;                    // 16 compute warps, producer, MMA issuer
constexpr int kCompute = 512;                    // compute threads
constexpr int kProducerWarp = 16;
constexpr int kMmaWarp = 17;
constexpr uint32_t kTileBytes = kT * kD * 2;     // 32 KB: two 16 KB boxes of 128 rows x 64 columns
constexpr uint32_t kColHalf = kTileBytes / 2;    // column-half stride of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxStages = 3;

struct Bars {
  uint64_t fixed_full;  // the CTA's fixed operands are in place
  uint64_t ring_full[kMaxStages];  // dK/dV pass: the Q ring; dQ pass: the (K, V) ring
  uint64_t ring_empty[kMaxStages];
  uint64_t do_full[2];  // dK/dV pass: the dO ring
  uint64_t do_empty[2];
  uint64_t s_full;    // S (S^T) computed
  uint64_t dp_full;   // dP (dP^T) computed
  uint64_t s_free;    // dQ pass: S and dP loaded by every compute thread
  uint64_t dp_free;   // dK/dV pass: dP^T loaded by every compute thread
  uint64_t p_full;    // dS written to shared memory (dK/dV pass: dS^T)
  uint64_t pt_full;   // dK/dV pass: P^T written to TMEM
  uint64_t ds_free;   // the MMA that read dS from shared memory completed
  uint64_t acc_full;
  uint64_t dq_full;   // fused pass: the dQ partial of one query tile is in TMEM
  uint64_t dq_free;   // fused pass: it was loaded by every compute thread
  uint64_t stg_full[2];  // fused pass: warpgroup x's (x = 0, 1) dQ block is staged
  uint64_t stg_free[2];  // fused pass: warpgroup x's staged block was read by the reducer
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok); }

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void init_bars(Bars* bars, int stages, uint32_t fixed_count) {
  mbar_init(&bars->fixed_full, fixed_count);
  for (int s = 0; s < stages; ++s) {
    mbar_init(&bars->ring_full[s], 1);
    mbar_init(&bars->ring_empty[s], 1);
  }
  mbar_init(&bars->s_full, 1);
  mbar_init(&bars->dp_full, 1);
  mbar_init(&bars->s_free, kCompute);
  mbar_init(&bars->dp_free, kCompute);
  mbar_init(&bars->p_full, kCompute);
  mbar_init(&bars->pt_full, kCompute);
  mbar_init(&bars->ds_free, 1);
  mbar_init(&bars->acc_full, 1);
  mbar_init(&bars->dq_full, 1);
  mbar_init(&bars->dq_free, kCompute);
  mbar_init(&bars->mma_done, 1);
  for (int s = 0; s < 2; ++s) {
    mbar_init(&bars->do_full[s], 1);
    mbar_init(&bars->do_empty[s], 1);
  }
  bars->abort = 0;
  fence_mbar_init();
}

// Loads one 128-row tile (two 64-column boxes) of `map` at row `row`.
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int x0, int row, int b,
                                          uint64_t pol) {
  tma_load_3d_hint(dst, map, bar, x0, row, b, pol);
  tma_load_3d_hint(dst + kColHalf, map, bar, x0 + 64, row, b, pol);
}

// D = A x B^T over K = 128, A and B 128-row K-major tiles in shared memory.
__device__ __forceinline__ void mma_ss_tile(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = (kk >> 2) * kColHalf + (kk & 3) * 32;
    mma_ss(d, sdesc_advance(da, off), sdesc_advance(db, off), idesc, (accumulate || kk > 0));
  }
}

// D (+)= A x B over K = 128, A a K-major tile in shared memory, B an MN-major tile [K rows][N = 128].
__device__ __forceinline__ void mma_ss_tile_mn(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  const uint64_t da = sdesc_sw128(a, 16, 1024), db = sdesc_sw128(b, kColHalf, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t a_off = (kk >> 2) * kColHalf + (kk & 3) * 32;
    mma_ss(d, sdesc_advance(da, a_off), sdesc_advance(db, kk * 2048), idesc,
           (accumulate || kk > 0));
  }
}

// D = A x B over K = 128, A and B MN-major tiles [K rows][M or N = 128] (A^T and B as stored).
__device__ __forceinline__ void mma_ss_tile_mnmn(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
  const uint64_t da = sdesc_sw128(a, kColHalf, 1024), db = sdesc_sw128(b, kColHalf, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    mma_ss(d, sdesc_advance(da, kk * 2048), sdesc_advance(db, kk * 2048), idesc,
           kk > 0);
  }
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

// Stores one 32-column chunk of a gradient row (fp32 accumulator values x mul).
__device__ __forceinline__ void store_grad_chunk(void* base, long long off, const uint32_t (&a)[32], float mul,
                                                 int mode) {
  if (mode == LCB_GRAD_BF16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(base) + off;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      uint4 v;
      v.x = pack_bf16x2(__uint_as_float(a[i]) * mul, __uint_as_float(a[i + 1]) * mul);
      v.y = pack_bf16x2(__uint_as_float(a[i + 2]) * mul, __uint_as_float(a[i + 3]) * mul);
      v.z = pack_bf16x2(__uint_as_float(a[i + 4]) * mul, __uint_as_float(a[i + 5]) * mul);
      v.w = pack_bf16x2(__uint_as_float(a[i + 6]) * mul, __uint_as_float(a[i + 7]) * mul);
      *reinterpret_cast<uint4*>(dst + i) = v;
    }
  } else {
    float* dst = static_cast<float*>(base) + off;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      float4 v = make_float4(__uint_as_float(a[i]) * mul, __uint_as_float(a[i + 1]) * mul,
                             __uint_as_float(a[i + 2]) * mul, __uint_as_float(a[i + 3]) * mul);
      if (mode == LCB_GRAD_F32_ACCUM) {
        // Added in L2, fire and forget: the epilogue does not wait for the old value, which in a ring
        // step's fp32 accumulator is rarely in L2. One CTA owns these rows in a launch, so the sum is
        // the plain fp32 add (subnormal sums flush to zero, as the atomic add does).
        asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + i), "f"(v.x), "f"(v.y), "f"(v.z),
                     "f"(v.w)
                     : "memory");
      } else {
        *reinterpret_cast<float4*>(dst + i) = v;
      }
    }
  }
}

// Zeroes `cols` values of a gradient row (overwrite modes only).
__device__ __forceinline__ void store_zero(void* base, long long off, int cols, int mode) {
  if (mode == LCB_GRAD_F32_ACCUM) return;
  if (mode == LCB_GRAD_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off);
    for (int i = 0; i < cols / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
    for (int i = 0; i < cols / 4; ++i) dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

__device__ __forceinline__ uint32_t start(Bars* bars, int stages, uint32_t fixed_count, int warp) {
  if (threadIdx.x == 0) init_bars(bars, stages, fixed_count);
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return bars->tmem_base;
}

__device__ __forceinline__ void teardown(uint32_t tbase, int warp) {
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// One-pass kernels: warp 18 adds the staged dQ blocks.
constexpr int kKvStages = 2;
constexpr int kFuThreads = 608;
constexpr int kFuReduceWarp = 18;
constexpr uint32_t kDqBlock = 128 * 32 * 4;  // one staged dQ block: 128 rows x 32 columns fp32
constexpr uint32_t kFuSmK = 0;
constexpr uint32_t kFuSmV = kTileBytes;
constexpr uint32_t kFuSmQ = 2 * kTileBytes;
constexpr uint32_t kFuSmDo = kFuSmQ + kKvStages * kTileBytes;
constexpr uint32_t kFuSmDs = kFuSmDo + kTileBytes;
constexpr uint32_t kFuSmStg = kFuSmDs + kTileBytes;
constexpr uint32_t kFuSmBar = kFuSmStg + 2 * kDqBlock;
constexpr uint32_t kFuSmStats = kFuSmBar + ((sizeof(Bars) + 15) & ~15u);  // per-warpgroup row statistics, 1 KB
constexpr uint32_t kFuSmem = kFuSmStats + 1024 + 1024;

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

}  // namespace
}  // namespace lcb
