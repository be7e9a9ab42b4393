// Rotary position embedding with several position axes: tokens of images and
// video carry a position per axis (time, height, width), and each of the 64
// feature pairs of a head turns by the position on its own axis,
//   a = pos[axis(k)][token] * theta^(-2k/128),  y_k + i y_{k+64} = e^{ia} (x_k + i x_{k+64}).
// The single-axis form is rope.cu's; this one is its counterpart for inputs
// whose positions are data (the caller's, on the device) rather than a range.
//
// Angles: the turn per unit of position, theta^(-2k/128) / 2 pi, is held as a
// 64-bit binary fraction, so pos * fraction modulo 2^64 is the angle modulo
// one turn by integer arithmetic alone, exact but for the fraction's own
// rounding (its 53 significant bits come from the host's double). An fp64
// product and its remainder (rope.cu's way) cost 2 fmod a lane, which for few
// heads is the whole time on a part with little fp64 throughput. The top of
// the fraction goes to fp32 and through sincospif; its rounding moves the
// angle by at most pi 2^-24.
//
// Bound by HBM (every element read and written once). One warp per token row,
// or per eight heads of one where rows are few: lane l owns pairs 2l, 2l + 1,
// forms their angles once, behind the loads of the first heads, and turns them
// in every head, eight heads' loads in flight before their stores (a call may
// be in place). 128K tokens x 32 heads: 320 us, 0.99 of the copy bandwidth (322
// us a call, back to back).
#include <cuda_bf16.h>

#include <algorithm>

#include "lcb_internal.h"

namespace lcb {
namespace {

constexpr int kD = 128;

// cos and sin of 2 pi * turn / 2^64.
__device__ __forceinline__ void turn64(unsigned long long turn, float& c, float& s) {
  const float x = __ll2float_rn(static_cast<long long>(turn)) * 1.0842021724855044e-19f;  // 2^-63: half turns in [-1, 1]
  sincospif(x, &s, &c);
}

template <class Pos>
__global__ void __launch_bounds__(256)
    rope_axes_kernel(const __nv_bfloat16* x, __nv_bfloat16* y, int B, int S, int H, long long rs, long long bs,
                     const Pos* __restrict__ pos, long long pas, long long pbs, long long prs, float sign, int per_warp,
                     const __grid_constant__ RopeAxes ax) {
  const int lane = threadIdx.x & 31;
  const int chunks = (H + per_warp - 1) / per_warp;
  const long long n = static_cast<long long>(B) * S * chunks;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  // The tables through shared memory: read straight from the parameters, each lane's own entry would be a constant
  // load apart, 32 in a row for every warp.
  __shared__ __align__(16) unsigned long long turn[kD / 2];
  __shared__ long long axis[kD / 2];
  if (threadIdx.x < kD / 2) {
    turn[threadIdx.x] = ax.turn[threadIdx.x];
    axis[threadIdx.x] = ax.axis[threadIdx.x] * pas;
  }
  __syncthreads();
  const unsigned long long g0 = turn[2 * lane], g1 = turn[2 * lane + 1];
  const long long a0 = axis[2 * lane], a1 = axis[2 * lane + 1];
  for (long long w = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); w < n; w += step) {
    const long long token = w / chunks;
    const int h0 = static_cast<int>(w - token * chunks) * per_warp, h1 = min(H, h0 + per_warp);
    const int b = static_cast<int>(token / S);
    const int s = static_cast<int>(token - static_cast<long long>(b) * S);
    const long long row = b * bs + static_cast<long long>(s) * rs + 2 * lane;
    uint32_t lo[8], hi[8];
    auto load = [&](int h) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (h + u < h1) {
          lo[u] = *reinterpret_cast<const uint32_t*>(x + row + (h + u) * kD);
          hi[u] = *reinterpret_cast<const uint32_t*>(x + row + (h + u) * kD + kD / 2);
        }
    };
    load(h0);
    const Pos* pr = pos + b * pbs + s * prs;
    float c0, s0, c1, s1;
    turn64(static_cast<unsigned long long>(static_cast<long long>(pr[a0])) * g0, c0, s0);
    turn64(static_cast<unsigned long long>(static_cast<long long>(pr[a1])) * g1, c1, s1);
    s0 *= sign;
    s1 *= sign;
    for (int h = h0;;) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (h + u < h1) {
          const float x0 = bf16lo_to_f32(lo[u]), x1 = bf16hi_to_f32(lo[u]);
          const float z0 = bf16lo_to_f32(hi[u]), z1 = bf16hi_to_f32(hi[u]);
          __nv_bfloat16* dst = y + row + (h + u) * kD;
          *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(x0 * c0 - z0 * s0, x1 * c1 - z1 * s1);
          *reinterpret_cast<uint32_t*>(dst + kD / 2) = pack_bf16x2(z0 * c0 + x0 * s0, z1 * c1 + x1 * s1);
        }
      if ((h += 8) >= h1) break;
      load(h);
    }
  }
}

}  // namespace

int launch_rope_axes(const void* x, void* y, int B, int S, int H, long long row_stride, long long batch_stride,
                     const void* pos, int pos_bytes, long long pos_axis_stride, long long pos_batch_stride,
                     long long pos_row_stride, int inverse, const RopeAxes& ax, cudaStream_t stream) {
  const long long rows = static_cast<long long>(B) * S;
  if (rows == 0) return 0;
  // A warp for eight heads where a warp a row would leave the GPU mostly empty (1031 rows x 8 heads: either way 3.2 us).
  const int per_warp = rows < 152 * 8 ? 8 : H;
  const long long warps = rows * ((H + per_warp - 1) / per_warp);
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((warps + 7) / 8, 152LL * 16));
  const __nv_bfloat16* xs = static_cast<const __nv_bfloat16*>(x);
  __nv_bfloat16* ys = static_cast<__nv_bfloat16*>(y);
  const float sign = inverse ? -1.f : 1.f;
  if (pos_bytes == 4)
    rope_axes_kernel<int><<<blocks, 256, 0, stream>>>(xs, ys, B, S, H, row_stride, batch_stride,
                                                      static_cast<const int*>(pos), pos_axis_stride, pos_batch_stride,
                                                      pos_row_stride, sign, per_warp, ax);
  else
    rope_axes_kernel<long long><<<blocks, 256, 0, stream>>>(xs, ys, B, S, H, row_stride, batch_stride,
                                                            static_cast<const long long*>(pos), pos_axis_stride,
                                                            pos_batch_stride, pos_row_stride, sign, per_warp, ax);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace lcb
