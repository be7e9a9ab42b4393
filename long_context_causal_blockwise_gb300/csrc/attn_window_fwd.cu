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
// product's A operand. The weights are 2^(s - m) against a reference m that is
// set to 2^16 above a row's largest score and raised lazily, only when a score
// passes that largest one by 24 to 31 in base 2. O / l is exact for any m; a
// tile's row sum of P stays below 2^15, so that l stays below 2^8 times the keys
// of the tiles that a row visits and O below that times max |v|, as in the full
// forward and the split kernel (a row that is finite in one form is finite in the
// others). Weights under 2^-126 are lost: 2^-110 of one that is there.
//
// What the window adds: a CTA streams only the key tiles that one of its rows
// can see (the sink tiles, then the window's), each query tile skips those of
// them that it does not see itself, and a tile needs the per-element mask only
// where the diagonal, the window's far edge, the last sink or the last key cuts
// it. Work is 4 * 128 flops a visible pair plus the hidden part of the cut
// tiles, at most two per query tile and edge.
//
// A CTA stays and walks over its share of the (head, 256 rows) items, each role
// on its own: the producer loads and the tensor core starts the next item while
// the epilogue warps still write the last one's O, so an item's start and end
// hide behind its neighbours.
//
// Where there are fewer items than half the SMs, a cluster of CTAs shares one:
// each takes an equal run of its visits, O, m and l stay in shared memory, and
// after the pass every CTA joins its share of the rows from all of them through
// distributed shared memory.
//
// What bounds it: the tensor core, fed from shared memory. Between an item's ends
// a visit of both query tiles takes 2350 cycles, 73 for each of its 32 products
// of 128 x 128 x 16 where the pipe alone needs 64; with a window of 1024 the ends
// are a sixth of an item. Measured on the way (us; 8K tokens x 32 heads, window
// 1024 / a 1000-row chunk of a 64K context, window 16384): 192 / 237 with a CTA
// per item and one thread issuing the products, 165 / 192 with the warp issuing
// them together (the descriptors stay in uniform registers), 140 / 193 with the
// epilogue in warps of its own and cut tiles in small loops, 128 / 178 with the
// maximum looked for only where a tile's sum says so, 122 / 170 with items
// decoded without the compiler's divisions, tile 0 beginning its next item beside
// tile 1's last visit and O stored in whole lines, 115 / 170 with loops for all
// code that runs a few times an item (one instruction fetch in six had missed).
// Splitting a row's columns over two warps (16 softmax warps) changed nothing.
//
//   warps 0-3   softmax of query tile 0 (thread = query row = TMEM lane)
//   warps 4-7   softmax of query tile 1
//   warps 8-11  epilogue of both
//   warp 12     TMA producer
//   warp 13     MMA issuer, owner of the TMEM allocation (14 and 15 fill the warpgroup)
//
// TMEM (512 columns x 128 lanes, fp32): S_0 [0,128), S_1 [128,256),
// O_0 [256,384), O_1 [384,512).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "attn_window.cuh"
#include "lcb_internal.h"
#include "mma_warp.cuh"

namespace cg = cooperative_groups;

namespace lcb {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kD = 128;
constexpr int kStages = 4;
constexpr int kThreads = 512;  // four warpgroups
constexpr int kEpilogueWarp = 8;
constexpr int kProducerWarp = 12;
constexpr int kMmaWarp = 13;
// Registers a thread: the block is launched with 128 each; the softmax
// warpgroups' 128 scores want more, and 2 * 168 + 2 * 88 = 4 * 128.
constexpr int kSoftmaxRegs = 168;
constexpr int kOtherRegs = 88;
constexpr uint32_t kTileBytes = kBN * kD * 2;  // 32 KB, two 16 KB halves of 64 columns
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr uint32_t kSmQ = 0;
constexpr uint32_t kSmKV = 2 * kTileBytes;
constexpr uint32_t kSmRow = kSmKV + kStages * kTileBytes;  // (m, l) of each query row
constexpr uint32_t kSmOut = kSmRow + 2 * kBM * 8;  // O on its way out: 128 bytes of each row of a tile
constexpr uint32_t kSmBar = kSmOut + kBM * 128;
// log2 units: the reference m lies kLead above the largest score when it is set; a score may pass it by
// kRescaleThreshold. Without the lead, raises are frequent for sharp scores (8K tokens, window 1024, scores of standard
// deviation 4: 226 us for 117; at 1.5 no difference).
constexpr float kLead = 16.0f;
constexpr float kRescaleThreshold = 8.0f;
constexpr long long kGroupBytes = 80LL << 20;  // K and V of the windows that a group of heads keeps in L2
constexpr int kSms = 152;

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[kStages];
  uint64_t kv_empty[kStages];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_full[2], o_free[2];
  uint64_t row_full[2], row_free[2];  // (m, l) of a finished query tile
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmemBytes = kSmBar + sizeof(Bars) + 1024;  // + alignment slack

// Division of 0 <= n < 2^31 by d >= 1, d known to the host: with 2^(s-1) < d <=
// 2^s and m = ceil(2^(31+s) / d) < 2^32, n m / 2^(31+s) exceeds n / d by less
// than n / 2^(31+s) < 1 / d, too little to reach the next integer. (The item
// decode below is between a CTA's items, where every cycle of it shows; the
// compiler's own division takes some 100.)
struct Divisor {
  uint32_t d, m, s;
  __host__ explicit Divisor(uint32_t by = 1) : d(by), s(0) {
    while ((1ull << s) < by) ++s;
    m = static_cast<uint32_t>(((1ull << (31 + s)) + by - 1) / by);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<unsigned long long>(static_cast<uint32_t>(n)) * m) >> (31 + s));
  }
};

struct Params {
  __nv_bfloat16* o;
  float* lse;
  long long o_rs, o_bs, l_hs, l_bs;
  int H, items;
  int parts;                             // CTAs of a cluster that share an item
  int nq;                                // items of a head
  int head_group, last_group, last_size;  // heads of a group; the last group, and its heads
  Divisor by_h, by_g, by_group_items, by_group, by_last;  // H, H / Hkv, nq * head_group, head_group, last_size
  WindowShape w;
  float scale_log2;
  DevStatus st;
};

constexpr uint32_t kWhere = 5u << 24;  // kernel id of timeout reports

// Item k of the grid's work: 256 query rows from q0 of head h of batch b.
// (b, h) pairs go in groups (as many as keep their windows' K and V in L2), a
// group's items query block by query block with its heads interleaved. Blocks
// come latest first, and first to last in every other group counted from the
// end: where the window spans much of the sequence later blocks cost more, and
// CTA c, which takes items c, c + 152, ..., then meets no jump between groups
// and ends on the cheap ones.
struct Item {
  int b, h, q0;
};

__device__ __forceinline__ Item item_of(const Params& p, int k) {
  const int group = p.by_group_items.div(k);
  const int within = k - group * p.nq * p.head_group;
  const bool last = group == p.last_group;  // it may be smaller
  const int at = last ? p.by_last.div(within) : p.by_group.div(within);
  const int bh = group * p.head_group + within - at * (last ? p.last_size : p.head_group);
  const int b = p.by_h.div(bh);
  return {b, bh - b * p.H, ((p.last_group - group) & 1 ? at : p.nq - 1 - at) * 2 * kBM};
}

// The visits of an item's two query tiles: `all` is the stream of key tiles that
// either one sees, of which [first, end) are this CTA's; query tile t takes part
// in those before sinks[t] and those of [from[t], to[t]).
template <bool kParts>
struct Visits {
  KeyTiles all, own[2];
  int first, end, sinks[2], from[2], to[2];
  // (no index that the compiler does not know: the arrays stay in registers)
  __device__ __forceinline__ bool any(int t) const {
    return kParts ? last(t) >= first : (t ? own[1].count() : own[0].count()) > 0;
  }
  __device__ __forceinline__ bool active(int t, int i) const {
    return t ? i < sinks[1] || (i >= from[1] && i < to[1]) : i < sinks[0] || (i >= from[0] && i < to[0]);
  }
  __device__ __forceinline__ int last(int t) const {
    return t ? (to[1] > from[1] ? to[1] : sinks[1]) - 1 : (to[0] > from[0] ? to[0] : sinks[0]) - 1;
  }
};

// Key tile kt in the stream `all`.
__device__ __forceinline__ int visit_of(const KeyTiles& all, int kt) {
  return kt <= all.ns ? kt : all.ns + kt - all.lo;
}

// The first of n visits that are part `part`'s.
__device__ __forceinline__ int part_begin(int n, int part, int parts) {
  return static_cast<int>(static_cast<long long>(n) * part / parts);
}

// How many of a query tile's own visits come before visit i of the stream.
__device__ __forceinline__ int visits_before(const KeyTiles& all, const KeyTiles& own, int i) {
  const int to = visit_of(all, own.hi);
  if (own.ns == own.lo) return min(i, to);  // one stretch
  return min(i, visit_of(all, own.ns)) + max(0, min(i, to) - visit_of(all, own.lo));
}

template <bool kParts>
__device__ __forceinline__ Visits<kParts> visits(const Params& p, int q0, int part) {
  Visits<kParts> v;
  v.all = key_tiles(p.w, q0, 2 * kBM);
  const int n = v.all.count();
  v.first = kParts ? part_begin(n, part, p.parts) : 0;
  v.end = kParts ? part_begin(n, part + 1, p.parts) : n;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const KeyTiles k = v.own[t] = key_tiles(p.w, q0 + t * kBM, kBM);
    v.sinks[t] = visit_of(v.all, k.ns);
    v.from[t] = visit_of(v.all, k.lo);
    v.to[t] = visit_of(v.all, k.hi);
    if (k.ns == k.lo) v.sinks[t] = v.to[t];  // one stretch
    if (kParts) {
      v.sinks[t] = min(v.sinks[t], v.end);
      v.from[t] = max(v.from[t], v.first);
      v.to[t] = min(v.to[t], v.end);
    }
  }
  return v;
}

// The columns of key tile kt that a query tile with own_ns sink tiles can use: all of a window
// tile's, a sink tile's up to the last sink. The second product runs over
// these alone, in steps of 16.
__device__ __forceinline__ int used_columns(const WindowShape& w, int own_ns, int kt) {
  return kt < own_ns ? min(kBN, w.sinks - kt * kBN) : kBN;
}

// Sets the reference m anew, kLead above the largest score `top`, where that
// passes it by more than the threshold, and rescales l and O (TMEM, 256 columns
// after S) with it. A row that has seen nothing yet takes its first: its l and O
// are 0.
__device__ __forceinline__ void raise_max(uint32_t tS, float& m, float& l, float top) {
  const bool fresh = m == -INFINITY;
  const bool resc = !fresh && top > m + kRescaleThreshold;
  const float m_new = top + kLead;
  if (__any_sync(0xffffffffu, resc)) {
    // O in pieces of 16 columns: beside the 128 scores, larger ones would not fit the registers
    const float alpha = resc ? ex2_approx(m - m_new) : 1.0f;
#pragma unroll 1
    for (int ch = 0; ch < 8; ++ch) {
      uint32_t o[16];
      tmem_ld_x16(tS + 256 + ch * 16, o);
#pragma unroll
      for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
      tmem_st_x16(tS + 256 + ch * 16, o);
    }
    if (resc) l *= alpha;
  }
  if (fresh || resc) m = m_new;
}

// P of 16 pairs of scores (bf16 pairs into pk), their sum into (s0, s1). P is
// rounded to bf16 for the second product (half a step, up to 2^-8 of each weight,
// of either sign); the sum is fp32.
__device__ __forceinline__ void weights(const uint32_t* s, uint32_t* pk, float c, float neg_m, float& s0, float& s1) {
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    float x0, x1;
    ffma2(x0, x1, __uint_as_float(s[2 * u]), __uint_as_float(s[2 * u + 1]), c, c, neg_m, neg_m);
    const float p0 = ex2_approx(x0);
    const float p1 = ex2_approx(x1);
    fadd2(s0, s1, s0, s1, p0, p1);
    pk[u] = pack_bf16x2(p0, p1);
  }
}

// The columns of a score tile that a row sees: [from, to], and those before
// `sink` up to `to`. A bit for each of the 32 from column ch on.
struct Seen {
  int from, to, sink;
  __device__ __forceinline__ uint32_t word(int ch) const {
    return low_bits(to + 1 - ch) & (~low_bits(from - ch) | low_bits(sink - ch));
  }
  // Whether it sees any of the tile's.
  __device__ __forceinline__ bool any() const { return to >= 0 && (from <= min(to, kBN - 1) || sink > 0); }
};

// 64 scores from column ch on, the hidden ones -inf.
__device__ __forceinline__ void load_seen(uint32_t (&s)[64], uint32_t tS, int ch, const Seen& v) {
  tmem_ld_x64(tS + ch, s);
  const uint32_t see[2] = {v.word(ch), v.word(ch + 32)};
#pragma unroll
  for (int k = 0; k < 64; ++k)
    if (!((see[k >> 5] >> (k & 31)) & 1u)) s[k] = __float_as_uint(-INFINITY);
}

// The same for 32.
__device__ __forceinline__ void load_seen(uint32_t (&s)[32], uint32_t tS, int ch, const Seen& v) {
  tmem_ld_x32(tS + ch, s);
  const uint32_t see = v.word(ch);
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (!((see >> k) & 1u)) s[k] = __float_as_uint(-INFINITY);
}

// A score tile in two passes: the maximum first, m raised if it has to be, then P
// over S in TMEM, l brought up. The second product reads columns [0, used).
// Columns go in pieces of 32, read again for the second pass (P overwrites only
// columns that were read before); a piece that no row of the warp sees costs
// only its zeros. Kept small: it runs for the first tile of a row and where the
// one-pass forms below give up.
__device__ __forceinline__ void softmax_two_pass(uint32_t tS, float c, float& m, float& l, const Seen v, int used,
                                                 bool keep_m) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int ch = 0; ch < used; ch += 32) {
    if (!__any_sync(0xffffffffu, v.word(ch))) continue;
    uint32_t s[32];
    load_seen(s, tS, ch, v);
    float m2[2] = {mx, -INFINITY};
#pragma unroll
    for (int e = 0; e < 32; e += 4)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        m2[u] = fmax3(m2[u], __uint_as_float(s[e + 2 * u]), __uint_as_float(s[e + 2 * u + 1]));
    mx = fmaxf(m2[0], m2[1]);
  }
  raise_max(tS, m, l, keep_m ? m : fmaxf(m, mx * c));
  const float neg_m = (m == -INFINITY) ? 0.f : -m;
  float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;  // sums of the even pieces, and of the odd
#pragma unroll 1
  for (int ch = 0; ch < used; ch += 32) {
    uint32_t pk[16];
    if (__any_sync(0xffffffffu, v.word(ch))) {
      uint32_t s[32];
      load_seen(s, tS, ch, v);
      weights(s, pk, c, neg_m, sa0, sa1);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) pk[k] = 0u;
    }
    tmem_st_x16_nowait(tS + ch / 2, pk);
    const float t0 = sa0, t1 = sa1;
    sa0 = sb0, sa1 = sb1, sb0 = t0, sb1 = t1;
  }
  tmem_wait_st();
  l += (sa0 + sb0) + (sa1 + sb1);
}

// The one-pass forms take P against the reference as it stands, without looking
// for a maximum: the tile's row sum tells afterwards whether a score was too far
// above it (some P over 2^15 makes a sum over 2^15; 128 P up to 2^8 make 2^15 at
// most). Then, or at a NaN, S is still in place and the two passes run; they
// keep the reference of a row whose own sum is fine. They run at once where the
// mask has shown some row of the warp nothing yet: a choice by position, so that
// no row's bits depend on another row's scores. (Where all that a row was shown
// had a score of -inf, its sum here is infinite or NaN, and it alone takes its
// first reference.) A row's first tile takes two passes because a weight of
// 2^-16, exact in bf16, for its largest score gives a row that sees one key that
// key's v to the bit; against 0 it would be a little faster, and would not.
// False: nothing was done.
constexpr float kMostSum = 32768.f;  // 2^15

// All 128 columns visible.
__device__ __forceinline__ bool softmax_whole(uint32_t tS, float c, float m, float& l, bool& fine) {
  uint32_t s[128], pk[64];
  tmem_ld_x64(tS, *reinterpret_cast<uint32_t(*)[64]>(s));
  tmem_ld_x64(tS + 64, *reinterpret_cast<uint32_t(*)[64]>(s + 64));
  float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q & 1)
      weights(s + 32 * q, pk + 16 * q, c, -m, sb0, sb1);
    else
      weights(s + 32 * q, pk + 16 * q, c, -m, sa0, sa1);
  }
  const float sum = (sa0 + sb0) + (sa1 + sb1);
  fine = sum <= kMostSum;
  if (!__all_sync(0xffffffffu, fine)) return false;
  tmem_st_x32_nowait(tS, *reinterpret_cast<uint32_t(*)[32]>(pk));
  tmem_st_x32_nowait(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
  tmem_wait_st();
  l += sum;
  return true;
}

// A tile that the mask cuts. The halves in a loop, not unrolled: this code runs
// a few times an item, and is fetched again each time.
__device__ __forceinline__ bool softmax_cut(uint32_t tS, float c, float m, float& l, const Seen v, int used,
                                            bool& fine) {
  uint32_t p0[32], p1[32];
  float sa0 = 0.f, sa1 = 0.f, sb0 = 0.f, sb1 = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) p1[k] = 0u;
#pragma unroll 1
  for (int ch = 0; ch < kBN; ch += 64) {
#pragma unroll
    for (int k = 0; k < 32; ++k) p0[k] = p1[k];
    if (ch < used && __any_sync(0xffffffffu, v.word(ch) | v.word(ch + 32))) {
      uint32_t s[64];
      load_seen(s, tS, ch, v);
      weights(s, p1, c, -m, sa0, sa1);
      weights(s + 32, p1 + 16, c, -m, sb0, sb1);
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) p1[k] = 0u;
    }
  }
  const float sum = (sa0 + sb0) + (sa1 + sb1);
  fine = sum <= kMostSum;
  if (!__all_sync(0xffffffffu, fine)) return false;
  tmem_st_x32_nowait(tS, p0);
  if (used > 64) tmem_st_x32_nowait(tS + 32, p1);
  tmem_wait_st();
  l += sum;
  return true;
}

// Piece `piece` (four floats) of a query row's O in shared memory, where parts are joined.
__device__ __forceinline__ float4* part_o(uint8_t* smem, int row, int piece) {
  return reinterpret_cast<float4*>(smem + kSmKV + row * (kD * 4) + ((piece ^ (row & 31)) << 4));
}

__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
}

// kParts: one item per cluster, its visits dealt to the cluster's CTAs.
template <bool kParts>
__global__ void __launch_bounds__(kThreads, 1)
    attn_window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  Bars* bars = reinterpret_cast<Bars*>(smem + kSmBar);
  volatile int* abort_flag = &bars->abort;
  const int warp = static_cast<int>(uniform(warp_id()));
  const int lane = static_cast<int>(lane_id());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 128);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->o_free[t], 128);
      mbar_init(&bars->row_full[t], 128);
      mbar_init(&bars->row_free[t], 128);
    }
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;

  const int part = kParts ? static_cast<int>(blockIdx.x) : 0;  // of item blockIdx.y

  // Every role walks the same items (the loops' bounds are written out each time: held in variables they cost the
  // issuing warp 6% of a long window's time); barrier phases carry on from one to
  // the next (ring slots by a running count, the others by one count per query tile).
  if (warp >= kProducerWarp) {
    regs_down();
    if (warp == kProducerWarp) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        const uint64_t pol = l2_policy_evict_last();
        int it = 0;              // K and V tiles loaded
        uint32_t nq[2] = {0, 0};  // Q tiles loaded
        bool ok = true;
        for (int k = static_cast<int>(kParts ? blockIdx.y : blockIdx.x); k < p.items && ok;
             k += kParts ? p.items : static_cast<int>(gridDim.x)) {
          const Item w = item_of(p, k);
          const Visits<kParts> v = visits<kParts>(p, w.q0, part);
          const int xq = w.h * kD, xk = p.by_g.div(w.h) * kD;
          // Q of tile 1 after the first K and V: its place is free last, and they must not wait for it.
          auto load_q = [&](int t) {
            if (!ok || !v.any(t)) return;
            ok = mbar_wait_inline(&bars->q_empty[t], (nq[t] & 1u) ^ 1u, abort_flag, p.st, kWhere | (7u << 16));
            if (!ok) return;
            mbar_arrive_expect_tx(&bars->q_full[t], kTileBytes);
            for (int half = 0; half < 2; ++half)
              tma_load_3d(smem + kSmQ + t * kTileBytes + half * kHalfBytes, &tm_q, &bars->q_full[t], xq + half * 64,
                          w.q0 + t * kBM, w.b);
            ++nq[t];
          };
          load_q(0);
          for (int i = v.first; i < v.end && ok; ++i) {
            for (int kv = 0; kv < 2; ++kv, ++it) {
              const int slot = it % kStages;
              const uint32_t ph = static_cast<uint32_t>(it / kStages) & 1u;
              if (!mbar_wait_inline(&bars->kv_empty[slot], ph ^ 1u, abort_flag, p.st, kWhere | (1u << 16))) {
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&bars->kv_full[slot], kTileBytes);
              const CUtensorMap* map = kv == 0 ? &tm_k : &tm_v;
              for (int half = 0; half < 2; ++half)
                tma_load_3d_hint(smem + kSmKV + slot * kTileBytes + half * kHalfBytes, map, &bars->kv_full[slot],
                                 xk + half * 64, v.all.tile(i) * kBN, w.b, pol);
            }
            if (i == v.first) load_q(1);
          }
        }
        if (!ok) {
          // Let every copy already issued land before the CTA can exit.
          for (int t = 0; t < 2; ++t)
            if (nq[t] > 0) drain_wait(&bars->q_full[t], (nq[t] - 1) & 1u, p.st.limit);
          for (int j = max(0, it - kStages); j < it; ++j)
            drain_wait(&bars->kv_full[j % kStages], static_cast<uint32_t>(j / kStages) & 1u, p.st.limit);
        }
      }
      __syncwarp();
    } else if (warp == kMmaWarp) {
      // ------------------------------------------------------------ MMA issuer
      // All lanes walk the loop, one elected lane issues.
      const uint32_t one = elect_one();
      const uint32_t tm = uniform(tbase);
      const uint32_t idesc_qk = idesc_bf16(kBM, kBN, false, false);
      const uint32_t idesc_pv = idesc_bf16(kBM, kD, false, true);
      const uint64_t q_desc = sdesc_sw128(sbase + kSmQ, 16, 1024);
      const uint64_t k_desc = sdesc_sw128(sbase + kSmKV, 16, 1024);
      const uint64_t v_desc = sdesc_sw128(sbase + kSmKV + kTileBytes, kHalfBytes, 1024);
      // Visit g of the CTA has K in ring slot 2 (g & 1) and V in the slot after it.
      auto issue_qk = [&](int t, uint32_t g) {
        const uint64_t qa = sdesc_advance(q_desc, t * kTileBytes);
        const uint64_t kb = sdesc_advance(k_desc, (g & 1u) * 2 * kTileBytes);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kHalfBytes + (kk & 3) * 32;
          mma_ss_if(tm + t * 128, sdesc_advance(qa, off), sdesc_advance(kb, off), idesc_qk, kk > 0, one);
        }
        tc_commit_if(&bars->s_full[t], one);
      };
      auto issue_pv = [&](int t, uint32_t g, uint32_t acc, int cols) {
        const uint64_t vb = sdesc_advance(v_desc, (g & 1u) * 2 * kTileBytes);
        if (cols == kBN) {
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts_if(tm + 256 + t * 128, tm + t * 128 + kk * 8, sdesc_advance(vb, kk * 2048), idesc_pv,
                      kk > 0 ? 1u : acc, one);
        } else {
#pragma unroll 1
          for (int kk = 0; kk * 16 < cols; ++kk)
            mma_ts_if(tm + 256 + t * 128, tm + t * 128 + kk * 8, sdesc_advance(vb, kk * 2048), idesc_pv,
                      kk > 0 ? 1u : acc, one);
        }
      };
      auto wait_kv = [&](uint32_t g, int v) {
        const bool r = mbar_wait_warp(&bars->kv_full[2 * (g & 1u) + v], (g >> 1) & 1u, abort_flag, p.st,
                                      kWhere | (3u << 16));
        tc_fence_after();
        return r;
      };
      uint32_t g = 0;  // visits of the items before, and of this one
      uint32_t q_phase = 0, p_phase = 0, o_phase = 0, acc = 0;  // bit t
      bool ok = true;
      auto wait_p = [&](int t) {
        ok = mbar_wait_warp(&bars->p_full[t], (p_phase >> t) & 1u, abort_flag, p.st, kWhere | (4u << 16));
        p_phase ^= 1u << t;
        if (ok && ((acc >> t) & 1u) == 0) {  // the first P V of an item writes over O: the previous one's has been read
          ok = mbar_wait_warp(&bars->o_free[t], ((o_phase >> t) & 1u) ^ 1u, abort_flag, p.st, kWhere | (8u << 16));
          o_phase ^= 1u << t;
        }
        tc_fence_after();
        return ok;
      };
      int k = static_cast<int>(kParts ? blockIdx.y : blockIdx.x) - (kParts ? p.items : static_cast<int>(gridDim.x));
      Visits<kParts> v;
      v.first = v.end = 0;
      for (bool more = true; more && ok;) {
        if (v.first < v.end) {
          for (int i = v.first; i + 1 < v.end && ok; ++i, ++g) {
            ok = wait_kv(g, 1);
            if (!ok) break;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok) continue;
              if (v.active(t, i)) {
                if (!wait_p(t)) continue;
                issue_pv(t, g, (acc >> t) & 1u, used_columns(p.w, (t ? v.own[1].ns : v.own[0].ns), v.all.tile(i)));
                acc |= 1u << t;
                if (i == v.last(t)) tc_commit_if(&bars->o_full[t], one);
              }
              if (v.active(t, i + 1)) {  // S over P once the product above has read it (issue order)
                if (!k_ready) {
                  ok = wait_kv(g + 1, 0);
                  if (!ok) continue;
                  k_ready = true;
                }
                issue_qk(t, g + 1);
                if (i + 1 == v.last(t)) tc_commit_if(&bars->q_empty[t], one);
              }
            }
            if (!ok) break;
            tc_commit_if(&bars->kv_empty[2 * (g & 1u) + 1], one);
            tc_commit_if(&bars->kv_empty[2 * ((g + 1) & 1u)], one);
          }
          if (!ok) break;
        }
        Visits<kParts> next;  // of the next item with a key, found while the softmax warps are at work
        do {
          k += kParts ? p.items : static_cast<int>(gridDim.x);
          more = k < p.items;
          if (more) next = visits<kParts>(p, item_of(p, k).q0, part);
        } while (more && next.first == next.end);
        if (v.first < v.end) ok = wait_kv(g, 1);
        // The item's last visit and the next one's first products: tile 0's go before the wait for tile 1's last P.
        const uint32_t g1 = v.first < v.end ? g + 1 : g;
        bool k_ready = false;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (!ok) continue;
          if (v.first < v.end && v.active(t, v.end - 1)) {  // in a loop: this code runs once an item
            if (!wait_p(t)) continue;
            const int cols = used_columns(p.w, (t ? v.own[1].ns : v.own[0].ns), v.all.tile(v.end - 1));
            const uint64_t vb = sdesc_advance(v_desc, (g & 1u) * 2 * kTileBytes);
#pragma unroll 1
            for (int kk = 0; kk * 16 < cols; ++kk)
              mma_ts_if(tm + 256 + t * 128, tm + t * 128 + kk * 8, sdesc_advance(vb, kk * 2048), idesc_pv,
                        kk > 0 ? 1u : (acc >> t) & 1u, one);
            tc_commit_if(&bars->o_full[t], one);
          }
          acc &= ~(1u << t);
          if (!more || !next.any(t)) continue;
          if (!k_ready) {
            ok = wait_kv(g1, 0);
            if (!ok) continue;
            k_ready = true;
          }
          ok = mbar_wait_warp(&bars->q_full[t], (q_phase >> t) & 1u, abort_flag, p.st, kWhere | (2u << 16));
          if (!ok) continue;
          q_phase ^= 1u << t;
          tc_fence_after();
          if (next.active(t, next.first)) {
            issue_qk(t, g1);
            if (next.last(t) == next.first) tc_commit_if(&bars->q_empty[t], one);
          }
        }
        if (!ok) break;
        if (v.first < v.end) tc_commit_if(&bars->kv_empty[2 * (g & 1u) + 1], one);
        if (more) tc_commit_if(&bars->kv_empty[2 * (g1 & 1u)], one);
        g = g1;
        v = next;
      }
      // Every MMA issued must finish before TMEM is released.
      tc_commit_if(&bars->mma_done, one);
      drain_wait(&bars->mma_done, 0, p.st.limit);
      __syncwarp();
    }
  } else if (warp >= kEpilogueWarp) {
    // ------------------------------------------------------------ epilogue
    regs_down();
    const int row = 32 * (warp - kEpilogueWarp) + lane;
    const uint32_t tO = tbase + 256 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if constexpr (kParts) {
      // This part's O, not divided by l yet, over the ring once nothing reads it any more, 16-byte pieces of a row
      // exchanged by the row's number (a warp writes a column of pieces, and reads a row). (m, l) are there already.
      const Visits<kParts> v = visits<kParts>(p, item_of(p, static_cast<int>(blockIdx.y)).q0, part);
      bool ok = true;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (v.any(t))
          ok = ok && mbar_wait_warp(&bars->row_full[t], 0, abort_flag, p.st, kWhere | (10u << 16)) &&
               mbar_wait_warp(&bars->o_full[t], 0, abort_flag, p.st, kWhere | (6u << 16));
        else
          reinterpret_cast<float2*>(smem + kSmRow)[t * kBM + row] = make_float2(-INFINITY, 0.f);
      }
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok || !v.any(t)) continue;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t o[32];
          tmem_ld_x32(tO + t * 128 + ch * 32, o);
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *part_o(smem, t * kBM + row, ch * 8 + j / 4) =
                make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), __uint_as_float(o[j + 2]),
                            __uint_as_float(o[j + 3]));
        }
      }
    } else {
      // O of a finished query tile out of TMEM while the softmax warps are on the next item.
      uint32_t phases = 0;  // bit t
      bool ok = true;
      for (int k = static_cast<int>(kParts ? blockIdx.y : blockIdx.x); k < p.items && ok;
           k += kParts ? p.items : static_cast<int>(gridDim.x)) {
        const Item w = item_of(p, k);
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if (!ok) continue;
          const int qi = w.q0 + t * kBM + row;
          const bool valid = qi < p.w.Sq;
          const bool any = key_tiles(p.w, w.q0 + t * kBM, kBM).count() > 0;  // else O was never formed
          float m = -INFINITY, l = 0.f;
          if (any) {
            ok = mbar_wait_warp(&bars->row_full[t], (phases >> t) & 1u, abort_flag, p.st, kWhere | (10u << 16));
            if (!ok) continue;
            const float2 r = reinterpret_cast<const float2*>(smem + kSmRow)[t * kBM + row];
            m = r.x;
            l = r.y;
            mbar_arrive(&bars->row_free[t]);
            ok = mbar_wait_warp(&bars->o_full[t], (phases >> t) & 1u, abort_flag, p.st, kWhere | (6u << 16));
            if (!ok) continue;
            phases ^= 1u << t;
            tc_fence_after();
          }
          const float inv_l = l == 0.f ? 0.f : 1.f / l;
          // Half of the columns at a time through shared memory, so that a store covers four whole lines, not a piece
          // of 32: the softmax warps' barrier arrivals wait behind them in the same queue.
          const int row0 = w.q0 + t * kBM + 32 * (warp - kEpilogueWarp);  // the warp's first
          __nv_bfloat16* dst = p.o + w.b * p.o_bs + static_cast<long long>(row0) * p.o_rs + w.h * kD;
          uint8_t* stage = smem + kSmOut + (warp - kEpilogueWarp) * 32 * 128;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t o[32];
            if (any) {
              tmem_ld_x32(tO + t * 128 + ch * 32, o);
              if (ch == 3) {
                tc_fence_before();
                mbar_arrive(&bars->o_free[t]);  // the next item's P V may write over O
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint4 u;
              u.x = pack_bf16x2(__uint_as_float(o[j]) * inv_l, __uint_as_float(o[j + 1]) * inv_l);
              u.y = pack_bf16x2(__uint_as_float(o[j + 2]) * inv_l, __uint_as_float(o[j + 3]) * inv_l);
              u.z = pack_bf16x2(__uint_as_float(o[j + 4]) * inv_l, __uint_as_float(o[j + 5]) * inv_l);
              u.w = pack_bf16x2(__uint_as_float(o[j + 6]) * inv_l, __uint_as_float(o[j + 7]) * inv_l);
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((((ch & 1) * 4 + j / 8) ^ (lane & 7)) << 4)) = u;
            }
            if (ch & 1) {
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = 4 * i + (lane >> 3);
                const uint4 u = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
                if (row0 + r < p.w.Sq)
                  *reinterpret_cast<uint4*>(dst + r * p.o_rs + (ch >> 1) * 64 + (lane & 7) * 8) = u;
              }
              __syncwarp();
            }
          }
          if (valid)
            p.lse[w.b * p.l_bs + w.h * p.l_hs + qi] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t tS = tbase + t * 128 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float c = p.scale_log2;
    uint32_t s_phase = 0, row_phase = 0;
    bool ok = true;
    for (int k = static_cast<int>(kParts ? blockIdx.y : blockIdx.x); k < p.items;
         k += kParts ? p.items : static_cast<int>(gridDim.x)) {
      const int q0 = item_of(p, k).q0 + t * kBM;
      const KeyTiles own = key_tiles(p.w, q0, kBM);
      int from = 0, to = own.count();  // of its visits, this CTA's
      if constexpr (kParts) {
        const KeyTiles all = key_tiles(p.w, q0 - t * kBM, 2 * kBM);
        from = visits_before(all, own, part_begin(all.count(), part, p.parts));
        to = visits_before(all, own, part_begin(all.count(), part + 1, p.parts));
      }
      float m = -INFINITY, l = 0.f;
      bool shown = false;  // whether the mask has left this row a key so far
      for (int i = from; i < to; ++i, s_phase ^= 1u) {
        ok = mbar_wait_warp(&bars->s_full[t], s_phase, abort_flag, p.st, kWhere | (5u << 16));
        if (!ok) break;
        tc_fence_after();
        const int kbase = own.tile(i) * kBN;
        const int p_first = p.w.pos0 + q0;
        const int pos = p_first + row;
        const Seen v = {pos - p.w.window + 1 - kbase, min(pos, p.w.Sk - 1) - kbase, p.w.sinks - kbase};
        const int used = used_columns(p.w, own.ns, own.tile(i));
        bool done = false, fine = false;
        if (__all_sync(0xffffffffu, shown)) {
          if (kbase + kBN - 1 <= p_first && kbase + kBN <= p.w.Sk &&
              (p_first + kBM - 1 - kbase < p.w.window || kbase + kBN <= p.w.sinks))
            done = softmax_whole(tS, c, m, l, fine);
          else
            done = softmax_cut(tS, c, m, l, v, used, fine);
        }
        if (!done) softmax_two_pass(tS, c, m, l, v, used, fine);
        shown |= v.any();
        tc_fence_before();
        mbar_arrive(&bars->p_full[t]);
      }
      if (ok && to > from) {  // m and l to the epilogue warps, and on to the next item
        ok = mbar_wait_warp(&bars->row_free[t], row_phase ^ 1u, abort_flag, p.st, kWhere | (9u << 16));
        if (!ok) break;
        row_phase ^= 1u;
        reinterpret_cast<float2*>(smem + kSmRow)[t * kBM + row] = make_float2(m, l);
        mbar_arrive(&bars->row_full[t]);
      }
      if (!ok) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
  if constexpr (kParts) {
    // What follows is every warp's: the warpgroups go back to the launch's 128 registers a thread (what two give up is
    // what the other two take).
    if (warp < kEpilogueWarp)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // Join the parts: row r = part + parts * i of the item's 256 here, i in turn by warp i % 16, lane = four features.
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    const Item w = item_of(p, static_cast<int>(blockIdx.y));
    const int rows = (min(2 * kBM, p.w.Sq - w.q0) - part + p.parts - 1) / p.parts;  // this CTA's
    float2* stats = reinterpret_cast<float2*>(smem + kSmRow);
    float2* ml = reinterpret_cast<float2*>(smem + kSmQ);  // [rows][parts] of (m, l)
    float* wt = reinterpret_cast<float*>(ml + 2 * kBM + kMaxCluster);  // and the parts' weights over the row's sum
    const int pair = threadIdx.x, i = pair / p.parts, c = pair - i * p.parts;
    if (i < rows) ml[pair] = *cluster.map_shared_rank(&stats[part + p.parts * i], c);
    __syncthreads();
    if (i < rows) {
      const float2* row = ml + i * p.parts;
      float M = -INFINITY, L = 0.f;
      for (int e = 0; e < p.parts; ++e) M = fmaxf(M, row[e].x);
      for (int e = 0; e < p.parts; ++e)
        if (row[e].y != 0.f) L += row[e].y * (row[e].x == M ? 1.f : ex2_approx(row[e].x - M));
      // negative: no weight in that part, and no O if none of its keys was visited
      wt[pair] = row[c].y == 0.f ? -1.f : (row[c].x == M ? 1.f : ex2_approx(row[c].x - M)) / L;
      if (c == 0)
        p.lse[w.b * p.l_bs + w.h * p.l_hs + w.q0 + part + p.parts * i] =
            L == 0.f ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
    }
    __syncthreads();
    const int pairs = (rows - warp + 15) / 16 * p.parts;  // (row, part) pairs of this warp, eight loads in flight
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    int li = warp, lc = 0, ai = warp, ac = 0;  // pair to load, pair to add
    for (int n = 0; n < pairs; n += 8) {
      float4 v[8];
      float f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        f[u] = n + u < pairs ? wt[li * p.parts + lc] : -1.f;
        v[u] = f[u] < 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                          : *cluster.map_shared_rank(part_o(smem, part + p.parts * li, lane), lc);
        if (++lc == p.parts) lc = 0, li += 16;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (n + u >= pairs) break;
        if (!(f[u] < 0.f))
          a = make_float4(a.x + f[u] * v[u].x, a.y + f[u] * v[u].y, a.z + f[u] * v[u].z, a.w + f[u] * v[u].w);
        if (++ac == p.parts) {
          uint2 o;
          o.x = pack_bf16x2(a.x, a.y);
          o.y = pack_bf16x2(a.z, a.w);
          const long long qi = w.q0 + part + p.parts * ai;
          *reinterpret_cast<uint2*>(p.o + w.b * p.o_bs + qi * p.o_rs + w.h * kD + lane * 4) = o;
          a = make_float4(0.f, 0.f, 0.f, 0.f);
          ac = 0;
          ai += 16;
        }
      }
    }
    cluster.sync();  // no CTA leaves while another reads its shared memory
  }
}

const void* parts_kernel() { return reinterpret_cast<const void*>(attn_window_fwd_kernel<true>); }
DeviceOnce g_parts_allowed;
ClusterCounts g_parts_resident;

cudaLaunchConfig_t parts_config(cudaLaunchAttribute* at, int parts, long long items, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(parts), static_cast<unsigned>(items));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = static_cast<unsigned>(parts);
  at->val.clusterDim.y = 1;
  at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

// Items, the parts that an item is dealt to, and an estimate of the time in us
// from measurements at 4 to 64 items: a visit takes 1.2 where one query tile has
// rows, 1.3 where both do, an item's start and end 5.4, a cluster and its join 5
// or 9 more (64 or 128 KB of O a CTA through distributed shared memory). The
// cluster, all of them resident at once, that promises most. us by parts 1, 2,
// 4, 8, 12, 16, 4 heads x 256 rows: window 16384 165, 103, 59, 38, 32, 30 (31 with
// the 15 that the estimate takes); 2048 32, 26, 20, 19, 19, 19; 512 17, 18, 16,
// 15, 16, 17.
struct Plan {
  long long items;
  int parts;
  double us;
};

Plan plan_of(const WindowShape& w, int B, int H) {
  Plan d = {static_cast<long long>((w.Sq + 2 * kBM - 1) / (2 * kBM)) * B * H, 1, 0.};
  const int visits = key_tiles(w, (w.Sq - 1) / (2 * kBM) * 2 * kBM, 2 * kBM).count();
  const double visit_us = w.Sq > kBM ? 1.3 : 1.18;
  d.us = 0.6 + std::ceil(static_cast<double>(d.items) / kSms) * (5.4 + (d.items > kSms ? 1.18 : visit_us) * visits);
  if (2 * d.items > kSms) return d;
  const ContextKey at = current_context();
  for (int c = 2; c <= kMaxCluster && c * d.items <= kSms; ++c) {
    const double us = (w.Sq > kBM ? 15. : 11.) + visit_us * ((visits + c - 1) / c);
    if (us < d.us &&
        resident_clusters(g_parts_resident, at, g_parts_allowed, parts_kernel(), kThreads, kSmemBytes, c) >= d.items)
      d.parts = c, d.us = us;
  }
  return d;
}

}  // namespace

int launch_window_fwd(const WindowFwd& a, cudaStream_t stream) {
  CUtensorMap tq, tk, tv;
  int rc;
  if ((rc = make_tma_map_bf16(&tq, a.q, a.B, a.w.Sq, a.H * kD, kBM)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tk, a.k, a.B, a.w.Sk, a.Hkv * kD, kBN)) != 0) return rc;
  if ((rc = make_tma_map_bf16(&tv, a.v, a.B, a.w.Sk, a.Hkv * kD, kBN)) != 0) return rc;
  Params p;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_rs = a.o_row_stride;
  p.o_bs = a.o_batch_stride;
  p.l_hs = a.lse_head_stride;
  p.l_bs = a.lse_batch_stride;
  p.H = a.H;
  p.by_g = Divisor(a.H / a.Hkv);
  p.w = a.w;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.st = a.st;
  const Plan plan = plan_of(a.w, a.B, a.H);
  if (plan.items > 0x7fffffffLL - kSms) return -1;
  p.items = static_cast<int>(plan.items);
  p.nq = (a.w.Sq + 2 * kBM - 1) / (2 * kBM);
  p.parts = plan.parts;
  const long long window_rows = std::min<long long>(a.w.Sk, static_cast<long long>(a.w.window) + a.w.sinks + 2 * kBM);
  const long long kv_heads = std::max<long long>(1, kGroupBytes / (window_rows * 4 * kD));
  const int heads = static_cast<int>(plan.items / p.nq);
  p.head_group = static_cast<int>(std::min<long long>(heads, kv_heads * (a.H / a.Hkv)));
  p.last_group = (heads - 1) / p.head_group;
  p.last_size = heads - p.last_group * p.head_group;
  p.by_h = Divisor(a.H);
  p.by_group_items = Divisor(p.nq * p.head_group);
  p.by_group = Divisor(p.head_group);
  p.by_last = Divisor(p.last_size);
  if (plan.parts > 1) {
    if ((rc = allow_clusters_once(g_parts_allowed, parts_kernel(), kSmemBytes)) != 0) return rc;
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = parts_config(&at, plan.parts, plan.items, stream);
    return cudaLaunchKernelEx(&cfg, attn_window_fwd_kernel<true>, tq, tk, tv, p) == cudaSuccess ? 0 : -4;
  }
  static DeviceOnce smem_set;
  const void* fn = reinterpret_cast<const void*>(attn_window_fwd_kernel<false>);
  if ((rc = set_smem_limit_once(smem_set, fn, kSmemBytes)) != 0) return rc;
  attn_window_fwd_kernel<false>
      <<<static_cast<unsigned>(std::min<long long>(plan.items, kSms)), kThreads, kSmemBytes, stream>>>(tq, tk, tv, p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

double window_tiles_us(const WindowShape& w, int B, int H) { return plan_of(w, B, H).us; }
int window_tiles_parts(const WindowShape& w, int B, int H) { return plan_of(w, B, H).parts; }

}  // namespace lcb
