// The sliding window with sinks, as the windowed-attention kernels see it.
//
// Query row i stands at position p = pos0 + i; key j (0 <= j < Sk) is visible
// to it iff j <= p and (p - j < window or j < sinks). Sizes are bounded by the
// C-ABI layer (kWindowMaxRows) so that every sum of a position, a key index and
// the window below stays inside 32 bits.
#pragma once

#include <cuda_runtime.h>

namespace lcb {

constexpr int kWindowMaxRows = 1 << 28;    // Sq, Sk, |pos0|
constexpr int kWindowMaxWindow = 1 << 30;  // a wider window hides nothing more: p - j < 2^29 + 1

struct WindowShape {
  int Sq, Sk, pos0, window, sinks;  // sinks <= Sk
};

// The key tiles (128 keys) that query rows [r0, r0 + rows) visit: sink tiles
// [0, ns) and window tiles [lo, hi), ns <= lo <= hi.
struct KeyTiles {
  int ns, lo, hi;
  __host__ __device__ int count() const { return ns + hi - lo; }
  // key tile of visit i
  __host__ __device__ int tile(int i) const { return i < ns ? i : lo + i - ns; }
};

__host__ __device__ inline KeyTiles key_tiles(const WindowShape& w, int r0, int rows) {
  KeyTiles k = {0, 0, 0};
  const int last = (r0 + rows < w.Sq ? r0 + rows : w.Sq) - 1;
  if (r0 >= w.Sq) return k;
  const int p_lo = w.pos0 + r0, p_hi = w.pos0 + last;
  if (p_hi < 0 || w.Sk == 0) return k;
  const int first = p_lo - w.window + 1;  // oldest key in any row's window
  const int end = p_hi + 1 < w.Sk ? p_hi + 1 : w.Sk;
  k.lo = first > 0 ? first / 128 : 0;
  k.hi = (first > 0 ? first : 0) < end ? (end + 127) / 128 : k.lo;
  const int sinks = w.sinks < end ? w.sinks : end;
  k.ns = (sinks + 127) / 128;
  if (k.hi == k.lo)  // no key in any window: the sinks alone
    k.lo = k.hi = k.ns;
  else if (k.ns > k.lo)
    k.ns = k.lo;
  return k;
}

// The query tiles [lo, hi) (128 rows from row 0) with a row that sees a key of
// tile kt: from the diagonal to the window's reach, or to the last row where
// the tile holds a sink.
struct QueryTiles {
  int lo, hi;
};

__host__ __device__ inline QueryTiles query_tiles(const WindowShape& w, int kt) {
  QueryTiles q = {0, 0};
  const int first_key = kt * 128;
  const int last_key = (first_key + 128 < w.Sk ? first_key + 128 : w.Sk) - 1;
  const int from = first_key - w.pos0 > 0 ? first_key - w.pos0 : 0;  // first row at or past the first key
  int to = w.Sq - 1;                                                 // last row that sees the last key
  if (first_key >= w.sinks && last_key - w.pos0 + (w.window - 1) < to) to = last_key - w.pos0 + (w.window - 1);
  if (from > to) return q;
  q.lo = from / 128;
  q.hi = to / 128 + 1;
  return q;
}

// How the one-pass backward is dealt out: key tile kt of a K/V head visits
// G * (hi - lo) (query head, query tile) pairs, cut into `segs` runs of equal
// length, one CTA each. Sink tiles (kt < sink_tiles) may have another number
// of runs than the others. Where there is more than one, every run's dK and dV
// go to a slot of fp32 partials, summed in order afterwards.
struct WindowBwdPlan {
  int key_tiles, sink_tiles, sink_segs, segs;
  long long sink_ctas, ctas;    // CTAs of the sink tiles (they come first), and of all
  long long slots;              // fp32 partials (dK and dV, 128 x 128 each)
  __host__ __device__ bool split(bool sink) const { return (sink ? sink_segs : segs) > 1; }
};

}  // namespace lcb
