// Gated linear recurrence s_t = a_t s_{t-1} + m_t x_t, forward and backward, and
// its single-token step.
//
// A tile is fwd_tile or bwd_tile tokens of one sequence by CT channels, a workgroup's work.
// Its threads are LX lanes across the channels (VEC each, one 16-byte load a
// token) by LY groups along the tokens; a group's L tokens stay in registers.  The
// recurrence is affine in the state, so a group folds its tokens into
// s_out = A s_in + S, the groups are composed in order through LDS by one thread
// per channel, and each group runs its tokens again from its own starting state.
// The backward needs the states before each token and the reverse recurrence
//   ds_t = dy_t + e_{t+1},  e_t = a_t ds_t,  e_{T+1} = dht
// which folds the same way (e_out = A e_in + E with the same A), so it reads
// the inputs once and recomputes the states from the tile's starting state that
// the forward left in the workspace.
//
// Between tiles: a single-pass scan with decoupled look-back (Merrill and Garland, 2016),
// in two levels.  Every tile publishes its fold (A, S); the last of each group of kGroup
// composes the group's folds, publishes the whole, looks back over the groups before
// it to the nearest whose end state is known, and publishes its own group's.  A tile
// takes that state through the folds of its own group; so the inputs cross HBM once
// and no tile waits for a chain of others to finish.  What a tile publishes of
// a channel is one 64-bit word, stored and loaded as one atomic access at device
// scope, so no fence is needed.  The workgroups of a channel tile take their tiles
// in an order (by a counter of that channel tile) in which a tile's predecessors
// were taken before it: they are running or done, and publish their folds without
// waiting for anybody, so every wait ends.  (Waits are
// bounded all the same: should the workspace be overwritten by someone else during
// the call, the states become NaN and the kernel ends.)
//
// What bounds it: HBM bytes (6 a channel and token forward, 10 backward, with bf16 and
// a gate per channel) while few sequences are long: then the tiles in flight, two
// workgroups a compute unit by registers, and what they wait for each other.  T = 32768,
// bf16, on a card whose large copy moves 4.9 TB/s:
//   4096 channels, a decay each:          184 us (4.4 TB/s), backward 278 us (4.8 TB/s)
//   16 heads of 128, softplus gate:       109 us (3.7 TB/s),          203 us (3.3 TB/s)
//   32 heads of 128, a decay per head, convex: 130 us (4.1 TB/s),     205 us (3.9 TB/s)
// and in fp32
//   16 heads of 128, softplus gate:       165 us (4.9 TB/s),          288 us (4.7 TB/s)
//   32 heads of 128, a decay per head, convex: 232 us (4.6 TB/s),     348 us (4.6 TB/s)
//   16 heads of 128, sigmoid gate, convex: 186 us (4.3 TB/s),         414 us (3.2 TB/s; spills)
// Without the look back (wrong results, timing alone) the softplus case took 103 and
// 167 us, and without its gate functions the forward took 102 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../gdr_device.h"
#include "../gdr_lds.h"
#include "gdr_gate.h"
#include "gdr_layer.h"
#include "gdr_wide.h"

namespace gdr {
namespace {

// Threads of a forward workgroup and of a backward one.
constexpr int kFwdThreads = 256, kBwdThreads = 256;

// ---- published words ----
// One 64-bit word per tile and channel: the high half is the fold's A, or one of
// two bit patterns (NaNs that put_fold never writes) that say that nothing is
// there yet or that the low half is the end state instead of the fold's S.
constexpr uint32_t kNothing = 0x7fffffffu, kState = 0x7ffffffeu;
constexpr int kMaxPolls = 1 << 20;

__device__ __forceinline__ void put(uint64_t* w, uint32_t hi, float lo) {
  __hip_atomic_store(w, (uint64_t(hi) << 32) | __float_as_uint(lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get(const uint64_t* w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_fold(uint64_t* w, float A, float S) {
  put(w, A != A ? 0x7fc00000u : __float_as_uint(A), S);
}
__device__ __forceinline__ void put_state(uint64_t* w, float s) { put(w, kState, s); }
__device__ __forceinline__ uint32_t hi_of(uint64_t w) { return uint32_t(w >> 32); }
__device__ __forceinline__ float lo_of(uint64_t w) { return __uint_as_float(uint32_t(w)); }

// The product p of decays of which `least` is the least.  If none is zero the product
// is not either: where it leaves fp32's range the least positive number stands for it,
// so that an infinite state before them is infinite after them, as token by token, and
// not 0 * inf = NaN.  A finite state gains 2^-149 of itself at most.
__device__ __forceinline__ float decay_product(float p, float least) {
  return p == 0.f && least != 0.f ? __uint_as_float(1) : p;
}

// Tiles of a sequence, counted from its start (its end, in the backward), form groups
// of kGroup.  A group's last tile, its leader, composes the group's folds and
// publishes the whole in its word; the state that reaches a group comes from the
// leaders before it, and a tile takes it through the folds of its own group, one by
// one.  Which sums are formed depends on the tiles' places alone, not on how far
// anybody was, and the states' front advances by up to kGroup groups per trip to
// memory.
// The size is a trade between few and many channels: T = 32768, bf16, forward and
// backward in us (the words are registers: the convex sigmoid backward spills 11, 17
// and 31 of them):
//   groups of                                    5         6         8
//   16 heads of 128, sigmoid gate, convex     120, 246  119, 255  123, 293
//   16 heads of 128, softplus gate            109, 203  108, 204  109, 205
//   2 heads of 128, softplus gate              27, 45    25, 42    22, 41
//   4096 channels, a decay each               184, 278  184, 277  183, 277
// Without groups, a tile looking back over eight tiles at a time, the 2 heads took 52, 95.
constexpr int kGroup = 6;

// The state after the nearest of `count` (at least one) groups: w + c is the nearest
// leader's word and each next one is `step` words on.
__device__ __forceinline__ float look_back(const uint64_t* w, int64_t step, int count, int c) {
  const int n = min(kGroup, count);
  uint64_t x[kGroup];
  for (int polls = 0;; ++polls) {
    // after the first try, two words a poll, the nearest fold (the last to come) and the
    // farthest state (the first): polling all words slows the stores waited for, to a
    // hundredth of the speed
    if (polls == 0 ||
        (hi_of(get(w + c)) != kNothing && hi_of(get(w + step * (n - 1) + c)) == kState)) {
      bool state = false, hole = false;
#pragma unroll
      for (int i = 0; i < kGroup; ++i) x[i] = get(w + step * min(i, n - 1) + c);
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        hole |= !state && hi_of(x[i]) == kNothing;
        state |= hi_of(x[i]) == kState;
      }
      if (state && !hole) break;
    }
    if (polls > kMaxPolls) return __builtin_nanf("");
    __builtin_amdgcn_s_sleep(4);
  }
  float s = 0.f;   // what lies beyond the nearest state is overwritten by it
#pragma unroll
  for (int i = kGroup - 1; i >= 0; --i)
    s = hi_of(x[i]) == kState ? lo_of(x[i]) : fmaf(__uint_as_float(hi_of(x[i])), s, lo_of(x[i]));
  return s;
}

// The state a tile of one channel starts from.  w: the tile's words; the tile before
// it is `step` words on; `pos` tiles come before it in its sequence and `left` after
// it; (A, S): its fold; init: the state the sequence starts from.
__device__ __forceinline__ float start_state(uint64_t* w, int64_t step, int pos, int left, int c, float init, float A,
                                             float S) {
  const int j = pos % kGroup, k = pos / kGroup;
  const bool leader = j == kGroup - 1 && left > 0;
  if (left > 0 && !leader) put_fold(w + c, A, S);
  if (pos == 0) return init;
  // x[i]: the tile i + 1 before this one
  uint64_t x[kGroup - 1];
  const uint64_t* head = w + step * (j + 1) + c;   // the leader of the group before
  float s = init;
  for (int polls = 0;; ++polls) {
    const bool wait_head = k > 0 && !leader;
    const uint64_t h = wait_head ? get(head) : 0;
    if (polls == 0 || (hi_of(get(w + step + c)) != kNothing && (!wait_head || hi_of(h) == kState))) {
      bool hole = wait_head && hi_of(h) != kState;
#pragma unroll
      for (int i = 0; i < kGroup - 1; ++i) x[i] = get(w + step * min(i + 1, max(j, 1)) + c);
#pragma unroll
      for (int i = 0; i < kGroup - 1; ++i) hole |= i < j && hi_of(x[i]) == kNothing;
      if (wait_head) s = lo_of(h);
      if (!hole) break;
    }
    if (polls > kMaxPolls) {
      if (leader) put_state(w + c, __builtin_nanf(""));
      return __builtin_nanf("");
    }
    __builtin_amdgcn_s_sleep(4);
  }
  if (leader) {
    float FA = 1.f, FS = 0.f, least = A;
#pragma unroll
    for (int i = kGroup - 2; i >= 0; --i) {
      const float a = __uint_as_float(hi_of(x[i]));
      FS = fmaf(a, FS, lo_of(x[i]));
      FA *= a;
      least = fminf(least, a);
    }
    FS = fmaf(A, FS, S);
    FA = decay_product(FA * A, least);
    if (k > 0) {
      put_fold(w + c, FA, FS);
      s = look_back(w + step * kGroup, step * kGroup, k, c);
    }
    put_state(w + c, fmaf(FA, s, FS));
    // read again rather than held: the look back needs the registers
#pragma unroll
    for (int i = 0; i < kGroup - 1; ++i) x[i] = get(w + step * (i + 1) + c);
  }
#pragma unroll
  for (int i = kGroup - 2; i >= 0; --i)
    if (i < j) s = fmaf(__uint_as_float(hi_of(x[i])), s, lo_of(x[i]));
  return s;
}

// VEC consecutive elements, 16 bytes (or one element): one access at the elements'
// own alignment, which the device allows, so that rows may start anywhere.
template <typename TIO, int VEC>
struct Vec {
  static_assert(VEC * sizeof(TIO) == 16, "16-byte vectors");
  typedef u32x4 Raw;
  typedef typename Wide<TIO>::T Any;
  static __device__ __forceinline__ Raw load(const TIO* b, uint32_t o) { return *reinterpret_cast<const Any*>(b + o); }
  static __device__ __forceinline__ void unpack(const Raw& u, float (&x)[VEC]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (VEC == 8) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(u[i]);
      }
    }
  }
  static __device__ __forceinline__ void store(TIO* b, uint32_t o, const float (&x)[VEC]) {
    Raw u;
    if constexpr (VEC == 8) {
      const uint2 lo = pack4_bf16(x[0], x[1], x[2], x[3]), hi = pack4_bf16(x[4], x[5], x[6], x[7]);
      u = Raw{lo.x, lo.y, hi.x, hi.y};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(x[i]);
    }
    *reinterpret_cast<Any*>(b + o) = u;
  }
};
template <typename TIO>
struct Vec<TIO, 1> {
  typedef float Raw;
  static __device__ __forceinline__ Raw load(const TIO* b, uint32_t o) { return IO<TIO>::load1(b, o); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[1]) { x[0] = r; }
  static __device__ __forceinline__ void store(TIO* b, uint32_t o, const float (&x)[1]) { IO<TIO>::store1(b, o, x[0]); }
};

// Geometry of a variant.
template <int VEC, int LX, int TH, int TT>
struct Geo {
  static constexpr int LY = TH / LX;
  static constexpr int L = TT / LY;       // tokens per thread
  static constexpr int CT = LX * VEC;     // channels per tile
  static_assert(CT <= TH && L >= 1, "a thread for every channel");
};

// Where a channel's values sit in a row of the LDS arrays: channel VEC x + v at v PV
// + x, so that a wave's threads write consecutive words (one v at a time), and PV and
// the row pitch are such that neither those writes (of 64 / LX rows) nor the reads of
// 64 consecutive channels of a row meet in the 64 banks.  Plain [LY][CT] rows cost the
// backward a fifth of its cycles in bank conflicts.
template <int VEC, int LX>
struct Cols {
  static constexpr int PV = VEC == 1 ? LX : VEC == 8 ? (LX == 16 ? 24 : 40) : (LX == 32 ? 48 : 80);
  static constexpr int PITCH = VEC * PV + (LX < 64 ? LX : 0);
  static __device__ __forceinline__ int at(int c) { return c % VEC * PV + c / VEC; }
};

// Channel tiles of CT channels or fewer: with one gate per head the whole heads that
// fit (the head's gate gradient is summed inside the workgroup), else CT.  Where
// rows do not start on a vector, tiles share the channels evenly instead, so that
// each has at least one vector's worth (a last vector overlaps the one before).
template <int GM>
__host__ __device__ __forceinline__ int channel_tiles(int CT, int C, int D) {
  const int step = GM == kScanHeadLog ? CT / D * D : CT;
  return (C + step - 1) / step;
}
template <int GM, bool WHOLE>
__device__ __forceinline__ void channel_tile(int CT, int C, int D, int nct, int ct, int& base, int& n) {
  if (!WHOLE) {
    base = int(int64_t(C) * ct / nct);
    n = int(int64_t(C) * (ct + 1) / nct) - base;
  } else {
    const int step = GM == kScanHeadLog ? CT / D * D : CT;
    base = ct * step;
    n = min(C - base, step);
  }
}

// The place of a tile (its row of the published words) in the order in which the
// workgroups take them, and the tile.  SAVED: tokens of a backward tile.
template <int TT, int SAVED>
__device__ __forceinline__ ScanTile tile_at(const ScanParams& p, int order, bool backward, int& row) {
  if (p.dense_T < 0) {
    row = backward ? p.NT - 1 - order : order;
    return p.tab[row];
  }
  // all sequences' first tiles, then all second ones, ...
  const int per = scan_tiles(p.dense_T, TT);
  const int level = order / p.N, seq = order - level * p.N, idx = backward ? per - 1 - level : level;
  row = seq * per + idx;
  const int saved = scan_tiles(p.dense_T, SAVED);
  return ScanTile{seq * p.dense_T + idx * TT, min(TT, p.dense_T - idx * TT), seq, idx, per - 1 - idx,
                  seq * saved + idx * (TT / SAVED)};
}

// The workgroup's place in the order of its channels' tiles: its number where no
// tile waits for another, else the next of the channel tile's counter.
__device__ __forceinline__ int take_order(const ScanParams& p, int ct, int nct, int* slot) {
  if (!p.words) return blockIdx.x / nct;
  if (threadIdx.x == 0) *slot = int(atomicAdd(p.counters + int64_t(ct) * kScanCounterStep, 1u));
  chain_barrier();
  return __builtin_amdgcn_readfirstlane(*slot);   // the same for all: keep it scalar
}

// decay_product for a thread's L tokens of VEC channels.  So few tokens seldom underflow:
// their decays are looked at again rather than kept track of.
template <int L, int VEC>
__device__ __forceinline__ void keep_nonzero(float (&A)[VEC], const float (&a)[L][VEC]) {
  bool any = false;
#pragma unroll
  for (int v = 0; v < VEC; ++v) any |= A[v] == 0.f;
  if (!any) return;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    bool zero = false;
#pragma unroll
    for (int i = 0; i < L; ++i) zero |= a[i][v] == 0.f;
    if (A[v] == 0.f && !zero) A[v] = __uint_as_float(1);
  }
}

// The gate of VEC channels: base-2 log decays, and what its gradient needs.
template <int VEC, int GM>
struct Gate {
  float eA[VEC], bias[VEC];
  __device__ __forceinline__ void init(const ScanParams& p, int c0) {
    if constexpr (GM == kScanSoftplus || GM == kScanSigmoid) {
      // heads of several channels hold whole vectors: one A_log a thread
      const float e0 = fast_exp2(p.A_log[c0 / p.D] * kLog2e);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        eA[v] = e0;
        bias[v] = p.dt_bias[c0 + v] * kLog2e;
      }
      if (p.D == 1) {
#pragma unroll
        for (int v = 1; v < VEC; ++v) eA[v] = fast_exp2(p.A_log[c0 + v] * kLog2e);
      }
    }
  }
  __device__ __forceinline__ float log2_decay(float g, int v, float gs) const {
    if constexpr (GM == kScanSoftplus) return gate_log2<0>(fmaf(g, kLog2e, bias[v]), eA[v], gs);
    else if constexpr (GM == kScanSigmoid) return gate_log2<1>(fmaf(g, kLog2e, bias[v]), eA[v], gs);
    else return g * kLog2e;
  }
};

// Raw gate values of row r of a tile: VEC of them, or the head's one.  `first`: the
// gate's first element of the tile.
template <typename TIO, int VEC, int GM>
struct GateRaw {
  typedef typename Vec<TIO, VEC>::Raw Raw;
  static __device__ __forceinline__ const TIO* first(const void* g, int64_t t, int C, int H) {
    return static_cast<const TIO*>(g) + t * C;
  }
  static __device__ __forceinline__ Raw load(const TIO* first, uint32_t r, int C, int H, int c0, int h) {
    return Vec<TIO, VEC>::load(first, r * C + c0);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&g)[VEC]) { Vec<TIO, VEC>::unpack(r, g); }
};
template <typename TIO, int VEC>
struct GateRaw<TIO, VEC, kScanHeadLog> {
  typedef float Raw;
  static __device__ __forceinline__ const TIO* first(const void* g, int64_t t, int C, int H) {
    return static_cast<const TIO*>(g) + t * H;
  }
  static __device__ __forceinline__ Raw load(const TIO* first, uint32_t r, int C, int H, int c0, int h) {
    return IO<TIO>::load1(first, r * H + h);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&g)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) g[v] = r;
  }
};

// First element of token row t of a [tokens][C] tensor.
template <typename TIO> __device__ __forceinline__ const TIO* row_at(const void* b, int64_t t, int C) {
  return static_cast<const TIO*>(b) + t * C;
}
template <typename TIO> __device__ __forceinline__ TIO* row_at(void* b, int64_t t, int C) {
  return static_cast<TIO*>(b) + t * C;
}

// Both kernels keep their loads in bounds without branches: rows past the tile's
// end and lanes past its channels load a valid neighbour's values, and the rows past
// the end are then made neutral (a = 1, no input), in a loop of its own that full
// tiles skip.  Barriers order LDS only.  A workgroup handles one tile; workgroups that
// stay and load their next tile's inputs ahead measured slower (117 us against 106 for
// the forward of T = 32768, 16 heads of 128: the registers halve the tile), as did
// three workgroups a compute unit (126 us: spills).
template <typename TIO, int VEC, int LX, int GM, bool CONVEX, bool WHOLE>
__global__ __launch_bounds__(kFwdThreads, 2) void k_scan_fwd(const ScanParams p) {
  constexpr int TT = fwd_tile(GM, LX * VEC > 128), kSaved = bwd_tile(GM, LX * VEC > 128, CONVEX);
  typedef Geo<VEC, LX, kFwdThreads, TT> G;
  typedef Vec<TIO, VEC> V;
  typedef GateRaw<TIO, VEC, GM> GR;
  typedef Cols<VEC, LX> K;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  __shared__ float sA[LY][K::PITCH], sS[LY][K::PITCH];
  __shared__ int slot;
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int nct = channel_tiles<GM>(CT, p.C, p.D), ct = blockIdx.x % nct;
  int cbase, nc;
  channel_tile<GM, WHOLE>(CT, p.C, p.D, nct, ct, cbase, nc);
  const int c = tid;   // the channel this thread composes
  const bool lead = c < nc;
  const bool on = lx * VEC < nc;
  const int v0 = min(lx * VEC, nc - VEC), c0 = cbase + v0;   // idle lanes repeat the last vector
  // LDS column of this thread's channel v, and of the channel it composes; whole vectors
  // (WHOLE) have columns of their own, overlapping ones share them
  auto col = [&](int v) { return WHOLE ? v * K::PV + lx : K::at(v0 + v); };
  const int cc = K::at(c);
  const int head = GM == kScanHeadLog ? c0 / p.D : 0;
  Gate<VEC, GM> gate;
  gate.init(p, c0);
  int row;
  const ScanTile tile = tile_at<TT, kSaved>(p, take_order(p, ct, nct, &slot), false, row);
  const int64_t sc = int64_t(tile.seq) * p.C + cbase + c;
  float s = 0.f;   // the tile's starting state, known to the lead threads
  if (tile.idx < kGroup && p.h0 && lead) s = p.h0[sc];
  if (tile.len == 0) {
    // a sequence without tokens: its state passes through
    if (lead && p.ht) p.ht[sc] = s;
    return;
  }
  typename GR::Raw rg[L];
  typename V::Raw rx[L];
  {
    const TIO* g = GR::first(p.g, tile.t_start, p.C, p.H);
    const TIO* x = row_at<TIO>(p.x, tile.t_start, p.C);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const uint32_t r = min(ly * L + i, tile.len - 1);
      rg[i] = GR::load(g, r, p.C, p.H, c0, head);
      rx[i] = V::load(x, r * p.C + c0);
    }
  }
  // the tokens' decays and, in the convex form, inputs (else they stay packed)
  float a[L][VEC], u[CONVEX ? L : 1][VEC];
  auto input = [&](int i, float (&x)[VEC]) {
    if constexpr (CONVEX) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[v] = u[i][v];
    } else {
      V::unpack(rx[i], x);
    }
  };
  {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float g[VEC];
      GR::unpack(rg[i], g);
      if constexpr (CONVEX) V::unpack(rx[i], u[i]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float l = gate.log2_decay(g[v], v, p.gate_scale);
        a[i][v] = fast_exp2(l);
        if constexpr (CONVEX) u[i][v] *= one_minus_exp2(l, a[i][v]);
      }
    }
  }
  if (tile.len < TT) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (ly * L + i >= tile.len) {
        rx[i] = {};
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          a[i][v] = 1.f;
          if constexpr (CONVEX) u[i][v] = 0.f;
        }
      }
  }
  {
    float A[VEC], S[VEC], x[VEC];
    input(0, S);
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = a[0][v];
#pragma unroll
    for (int i = 1; i < L; ++i) {
      input(i, x);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[v] = fmaf(a[i][v], S[v], x[v]);
        A[v] *= a[i][v];
      }
    }
    keep_nonzero<L, VEC>(A, a);
#pragma unroll
    for (int v = 0; v < VEC; ++v) { sA[ly][col(v)] = A[v]; sS[ly][col(v)] = S[v]; }
  }
  chain_barrier();
  // one thread per channel composes the groups, and publishes before it does more
  if (lead) {
    uint64_t* w = p.words + int64_t(row) * p.C + cbase;
    float At = 1.f, St = 0.f, least = 1.f;
#pragma unroll
    for (int y = 0; y < LY; ++y) {
      St = fmaf(sA[y][cc], St, sS[y][cc]);
      At *= sA[y][cc];
      least = fminf(least, sA[y][cc]);
    }
    At = decay_product(At, least);
    s = start_state(w, -int64_t(p.C), tile.idx, tile.after, c, s, At, St);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);   // the folds in LDS are read again, not held
    if (tile.after == 0 && p.ht) p.ht[sc] = fmaf(At, s, St);
    float* saved = p.carry + int64_t(tile.saved) * p.C + cbase + c;
#pragma unroll
    for (int y = 0; y < LY; ++y) {
      constexpr int kPer = kSaved / L;   // groups per backward tile
      static_assert(kPer * L == kSaved && TT % kSaved == 0, "saved states at group borders");
      if (y % kPer == 0 && y * L < tile.len) saved[int64_t(y / kPer) * p.C] = s;
      const float Sy = sS[y][cc];
      sS[y][cc] = s;
      s = fmaf(sA[y][cc], s, Sy);
    }
  }
  chain_barrier();
  TIO* out = row_at<TIO>(p.y, tile.t_start, p.C);
  float y[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) y[v] = sS[ly][col(v)];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int r = ly * L + i;
    float x[VEC];
    input(i, x);
#pragma unroll
    for (int v = 0; v < VEC; ++v) y[v] = fmaf(a[i][v], y[v], x[v]);
    if (on && r < tile.len) V::store(out, uint32_t(r) * p.C + c0, y);
  }
}

template <typename TIO, int VEC, int LX, int GM, bool CONVEX, bool WHOLE>
__global__ __launch_bounds__(kBwdThreads, 2) void k_scan_bwd(const ScanParams p) {
  constexpr int TT = bwd_tile(GM, LX * VEC > 128, CONVEX);
  typedef Geo<VEC, LX, kBwdThreads, TT> G;
  typedef Vec<TIO, VEC> V;
  typedef GateRaw<TIO, VEC, GM> GR;
  typedef Cols<VEC, LX> K;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  constexpr bool kPar = GM == kScanSoftplus || GM == kScanSigmoid;
  constexpr bool kLog = GM == kScanSoftplus || CONVEX;   // the logarithm is needed again
  __shared__ float sA[LY][K::PITCH], sS[LY][K::PITCH], sE[LY][K::PITCH];
  __shared__ float sG[GM == kScanHeadLog ? TT : 1][LX + 1];
  __shared__ int slot;
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int nct = channel_tiles<GM>(CT, p.C, p.D), ct = blockIdx.x % nct;
  int cbase, nc;
  channel_tile<GM, WHOLE>(CT, p.C, p.D, nct, ct, cbase, nc);
  const int c = tid;
  const bool lead = c < nc;
  const bool on = lx * VEC < nc;
  const int v0 = min(lx * VEC, nc - VEC), c0 = cbase + v0;   // idle lanes repeat the last vector
  // LDS column of this thread's channel v, and of the channel it composes; whole vectors
  // (WHOLE) have columns of their own, overlapping ones share them
  auto col = [&](int v) { return WHOLE ? v * K::PV + lx : K::at(v0 + v); };
  const int cc = K::at(c);
  const int head = GM == kScanHeadLog ? c0 / p.D : 0;
  Gate<VEC, GM> gate;
  gate.init(p, c0);
  int row;
  const ScanTile tile = tile_at<TT, TT>(p, take_order(p, ct, nct, &slot), true, row);
  // the state before the tile, and what the reverse recurrence brings from after it
  const int64_t sc = int64_t(tile.seq) * p.C + cbase + c;
  float* partial = p.part + int64_t(row) * 2 * p.C + cbase + c;
  float s0 = 0.f, e0 = 0.f;
  if (tile.after < kGroup && p.dht && lead) e0 = p.dht[sc];
  if (tile.len == 0) {
    if (lead && p.dh0) p.dh0[sc] = e0;
    if (kPar && lead) partial[0] = partial[p.C] = 0.f;
    return;
  }
  if (lead) s0 = p.carry[int64_t(tile.saved) * p.C + cbase + c];
  typename GR::Raw rg[L];
  typename V::Raw rx[L], rdy[L];
  {
    const TIO* g = GR::first(p.g, tile.t_start, p.C, p.H);
    const TIO* x = row_at<TIO>(p.x, tile.t_start, p.C);
    const TIO* dy = row_at<TIO>(p.dy, tile.t_start, p.C);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const uint32_t r = min(ly * L + i, tile.len - 1);
      rg[i] = GR::load(g, r, p.C, p.H, c0, head);
      rx[i] = V::load(x, r * p.C + c0);
      rdy[i] = V::load(dy, r * p.C + c0);
    }
  }
  // per token: the decay, its base-2 logarithm, the gate's slope, the input; `u`
  // becomes the state before the token
  float a[L][VEC], l[kLog ? L : 1][VEC], dz[kPar ? L : 1][VEC], u[L][VEC];
  {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float g[VEC];
      GR::unpack(rg[i], g);
      V::unpack(rx[i], u[i]);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float l2;
        if constexpr (kPar)
          gate_log2_grad<GM == kScanSoftplus ? 0 : 1>(fmaf(g[v], kLog2e, gate.bias[v]), gate.eA[v], p.gate_scale, l2,
                                                       dz[i][v]);
        else l2 = g[v] * kLog2e;
        a[i][v] = fast_exp2(l2);
        if constexpr (kLog) l[i][v] = l2;
        if constexpr (CONVEX) u[i][v] *= one_minus_exp2(l2, a[i][v]);
      }
    }
  }
  if (tile.len < TT) {
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (ly * L + i >= tile.len) {
        rdy[i] = {};
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          a[i][v] = 1.f;
          u[i][v] = 0.f;
          if constexpr (kPar) dz[i][v] = 0.f;
          if constexpr (kLog) l[i][v] = 0.f;
        }
      }
  }
  {
    float A[VEC], S[VEC], E[VEC], dy[VEC];
    V::unpack(rdy[L - 1], dy);
#pragma unroll
    for (int v = 0; v < VEC; ++v) { A[v] = a[0][v]; S[v] = u[0][v]; E[v] = a[L - 1][v] * dy[v]; }
#pragma unroll
    for (int i = 1; i < L; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[v] = fmaf(a[i][v], S[v], u[i][v]);
        A[v] *= a[i][v];
      }
#pragma unroll
    for (int i = L - 2; i >= 0; --i) {
      V::unpack(rdy[i], dy);
#pragma unroll
      for (int v = 0; v < VEC; ++v) E[v] = a[i][v] * (dy[v] + E[v]);
    }
    keep_nonzero<L, VEC>(A, a);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sA[ly][col(v)] = A[v];
      sS[ly][col(v)] = S[v];
      sE[ly][col(v)] = E[v];
    }
  }
  chain_barrier();
  if (lead) {
    uint64_t* w = p.words + int64_t(row) * p.C + cbase;
    float At = 1.f, Et = 0.f, least = 1.f;
#pragma unroll
    for (int y = LY - 1; y >= 0; --y) {
      Et = fmaf(sA[y][cc], Et, sE[y][cc]);
      At *= sA[y][cc];
      least = fminf(least, sA[y][cc]);
    }
    At = decay_product(At, least);
    e0 = start_state(w, p.C, tile.after, tile.idx, c, e0, At, Et);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);   // the folds in LDS are read again, not held
    if (tile.idx == 0 && p.dh0) p.dh0[sc] = fmaf(At, e0, Et);
#pragma unroll
    for (int y = LY - 1; y >= 0; --y) {
      const float Ey = sE[y][cc];
      sE[y][cc] = e0;
      e0 = fmaf(sA[y][cc], e0, Ey);
    }
#pragma unroll
    for (int y = 0; y < LY; ++y) {
      const float Sy = sS[y][cc];
      sS[y][cc] = s0;
      s0 = fmaf(sA[y][cc], s0, Sy);
    }
  }
  chain_barrier();
  float e[VEC], sumz[VEC], sumA[VEC];
  {
    float s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      s[v] = sS[ly][col(v)];
      e[v] = sE[ly][col(v)];
      sumz[v] = sumA[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float n = fmaf(a[i][v], s[v], u[i][v]);
        u[i][v] = s[v];
        s[v] = n;
      }
  }
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    const int r = ly * L + i;
    float dx[VEC], dg[VEC], x[VEC], dy[VEC], g[VEC];
    V::unpack(rdy[i], dy);
    if constexpr (CONVEX) V::unpack(rx[i], x);
    if constexpr (GM == kScanSigmoid) GR::unpack(rg[i], g);
    float dsum = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float ds = dy[v] + e[v];
      e[v] = a[i][v] * ds;
      float dl;
      if constexpr (CONVEX) {
        dl = e[v] * (u[i][v] - x[v]);
        dx[v] = one_minus_exp2(l[i][v], a[i][v]) * ds;
      } else {
        dl = e[v] * u[i][v];
        dx[v] = ds;
      }
      if constexpr (kPar) {
        // rows past the end add nothing, whatever state or gradient passes them (an
        // infinite one times their slope of zero would be a NaN in the sums)
        dl = r < tile.len ? dl : 0.f;
        dg[v] = dl * dz[i][v];
        // d lambda / d A_log: lambda, or the slope by z times z
        if constexpr (GM == kScanSoftplus)
          sumA[v] = fmaf(dl, fmaxf(l[i][v], -3.0e38f), sumA[v]);
        else
          sumA[v] = fmaf(dg[v], fminf(fmaxf(fmaf(g[v], kLog2e, gate.bias[v]), -3.0e38f), 3.0e38f), sumA[v]);
        sumz[v] += dg[v];
      } else {
        dg[v] = dl;
        dsum += dl;
      }
    }
    if (on && r < tile.len) {
      V::store(row_at<TIO>(p.dx, tile.t_start, p.C), uint32_t(r) * p.C + c0, dx);
      if constexpr (GM != kScanHeadLog) V::store(row_at<TIO>(p.dg, tile.t_start, p.C), uint32_t(r) * p.C + c0, dg);
    }
    if constexpr (GM == kScanHeadLog) sG[r][lx] = dsum;
  }
  if constexpr (GM == kScanHeadLog) {
    chain_barrier();
    const int heads = nc / p.D, lanes = p.D / VEC, h0 = cbase / p.D;
    for (int i = tid; i < tile.len * heads; i += kBwdThreads) {
      const int r = i / heads, h = i - r * heads;
      float d = 0.f;
      for (int m = 0; m < lanes; ++m) d += sG[r][h * lanes + m];
      IO<TIO>::store1(p.dg, (int64_t(tile.t_start) + r) * p.H + h0 + h, d);
    }
  }
  if constexpr (kPar) {
    chain_barrier();
#pragma unroll
    for (int v = 0; v < VEC; ++v) { sS[ly][col(v)] = sumz[v]; sE[ly][col(v)] = sumA[v]; }
    chain_barrier();
    if (lead) {
      float z = 0.f, zA = 0.f;
#pragma unroll
      for (int y = 0; y < LY; ++y) { z += sS[y][cc]; zA += sE[y][cc]; }
      partial[0] = z;
      partial[p.C] = zA * 0.6931471805599453f;   // lambda and z are in base-2 units
    }
  }
}

// ddt_bias and dA_log from the tiles' partial sums, in 64 bits and a fixed order.
// Many tiles are first summed in kParamSplit runs (64 channels a workgroup), so
// that the whole chip reads them: 8 us for 512 tiles of 2048 channels, 14 us with a
// workgroup per head alone.
__global__ __launch_bounds__(256) void k_scan_param_runs(const ScanParams p) {
  __shared__ double sz[256], sa[256];
  const int tid = threadIdx.x, c = blockIdx.x * 64 + (tid & 63), g = tid >> 6;
  const int r0 = int(int64_t(p.NT) * blockIdx.y / kParamSplit), r1 = int(int64_t(p.NT) * (blockIdx.y + 1) / kParamSplit);
  double z = 0.0, zA = 0.0;
  if (c < p.C) {
#pragma unroll 8
    for (int i = r0 + g; i < r1; i += 4) {
      const float* q = p.part + int64_t(i) * 2 * p.C + c;
      z += q[0];
      zA += q[p.C];
    }
  }
  sz[tid] = z;
  sa[tid] = zA;
  __syncthreads();
  if (g == 0 && c < p.C) {
    double* q = p.runs + int64_t(blockIdx.y) * 2 * p.C + c;
    q[0] = sz[tid] + sz[tid + 64] + sz[tid + 128] + sz[tid + 192];
    q[p.C] = sa[tid] + sa[tid + 64] + sa[tid + 128] + sa[tid + 192];
  }
}

// A workgroup per head (several narrow ones), its threads a row group each of the
// tiles or of their runs.
constexpr int kParamThreads = 1024;
__host__ __device__ __forceinline__ int param_heads(int D) { return D >= 64 ? 1 : 64 / D; }

template <typename T>
__global__ __launch_bounds__(kParamThreads) void k_scan_params(const ScanParams p, const T* rows, int n) {
  __shared__ double sz[kParamThreads], sa[kParamThreads];
  const int h0 = blockIdx.x * param_heads(p.D), heads = min(param_heads(p.D), p.H - h0);
  const int cw = heads * p.D, groups = kParamThreads / cw;
  const int tid = threadIdx.x, c = tid % cw, g = tid / cw;
  double z = 0.0, zA = 0.0;
  if (g < groups) {
    const T* q = rows + int64_t(h0) * p.D + c;
#pragma unroll 8
    for (int i = g; i < n; i += groups) {
      z += q[int64_t(i) * 2 * p.C];
      zA += q[int64_t(i) * 2 * p.C + p.C];
    }
  }
  sz[tid] = z;
  sa[tid] = zA;
  __syncthreads();
  if (g == 0) {
    for (int i = 1; i < groups; ++i) { z += sz[i * cw + c]; zA += sa[i * cw + c]; }
    p.ddt_bias[int64_t(h0) * p.D + c] = float(z);
    sa[c] = zA;
  }
  __syncthreads();
  if (tid < heads) {
    double d = 0.0;
    for (int i = 0; i < p.D; ++i) d += sa[tid * p.D + i];
    p.dA_log[h0 + tid] = float(d);
  }
}

// What a call's main kernel finds: the counters cleared and the words marked as not
// published, and the tile rows of up to kScanBatch sequences (workgroup i: sequence i),
// TT tokens a tile.
__global__ __launch_bounds__(256) void k_scan_prologue(uint32_t* counters, int nc, uint64_t* words, int64_t n,
                                                       ScanTile* tab, int TT, int saved, const ScanBatch b) {
  if (words) {
    const int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x, all = int64_t(gridDim.x) * 256;
    for (int64_t i = t; i < nc; i += all) counters[i * kScanCounterStep] = 0;
    ulonglong2* w = reinterpret_cast<ulonglong2*>(words);
    constexpr uint64_t kNo = uint64_t(kNothing) << 32;
    for (int64_t i = t; 2 * i < n; i += all) w[i] = ulonglong2{kNo, kNo};
  }
  const int i = blockIdx.x;
  if (i >= b.n) return;
  const int len = b.len[i], tiles = scan_tiles(len, TT);
  for (int j = threadIdx.x; j < tiles; j += 256)
    tab[b.tile0[i] + j] = ScanTile{b.t_start[i] + j * TT, min(TT, len - j * TT), b.seq0 + i, j, tiles - 1 - j,
                                   b.saved0[i] + j * (TT / saved)};
}

// One token a row: a workgroup takes 256 VEC channels of one row, and where later
// rows name the same slot, of those too, in order.
template <typename TIO, int VEC, int GM>
__global__ __launch_bounds__(256) void k_scan_step(const ScanStepParams p) {
  const int chunks = (p.C + 256 * VEC - 1) / (256 * VEC);
  int n = blockIdx.x / chunks;
  const int c0 = (int(blockIdx.x) - n * chunks) * 256 * VEC + int(threadIdx.x) * VEC;
  const int slot = p.slots ? p.slots[n] : n;
  if (slot < 0 || slot >= p.P) return;
  bool later = false;
  if (p.slots) {
    bool earlier = false;
    for (int m = threadIdx.x; m < p.N; m += 256)
      if (p.slots[m] == slot) {
        earlier |= m < n;
        later |= m > n;
      }
    if (__syncthreads_or(earlier)) return;
    later = __syncthreads_or(later);
  }
  if (c0 >= p.C) return;
  Gate<VEC, GM> gate;
  ScanParams q{};
  q.D = p.D; q.C = p.C; q.H = p.H; q.A_log = p.A_log; q.dt_bias = p.dt_bias; q.g = p.g;
  gate.init(q, c0);
  float s[VEC];
  float* st = p.state + int64_t(slot) * p.C + c0;
  if constexpr (VEC == 1) s[0] = st[0];
  else if constexpr (VEC == 4) IO<float>::load4(st, 0, s);
  else IO<float>::load8(st, 0, s);
  for (;;) {
    float g[VEC], x[VEC];
    typedef GateRaw<TIO, VEC, GM> GR;
    GR::unpack(GR::load(GR::first(p.g, n, p.C, p.H), 0, p.C, p.H, c0, GM == kScanHeadLog ? c0 / p.D : 0), g);
    Vec<TIO, VEC>::unpack(Vec<TIO, VEC>::load(row_at<TIO>(p.x, n, p.C), c0), x);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float l = gate.log2_decay(g[v], v, p.gate_scale);
      const float a = fast_exp2(l);
      s[v] = a * s[v] + (p.convex ? one_minus_exp2(l, a) * x[v] : x[v]);
    }
    Vec<TIO, VEC>::store(row_at<TIO>(p.y, n, p.C), c0, s);
    if (!later) break;
    do ++n; while (n < p.N && p.slots[n] != slot);
    if (n >= p.N) break;
  }
  if constexpr (VEC == 1) st[0] = s[0];
  else if constexpr (VEC == 4) IO<float>::store4(st, 0, s[0], s[1], s[2], s[3]);
  else IO<float>::store8(st, 0, s);
}

template <typename TIO, int VEC, int LX, int GM, bool CONVEX, bool WHOLE>
int launch_whole(const ScanParams& p, bool backward, hipStream_t s) {
  const dim3 grid(unsigned(int64_t(p.NT) * channel_tiles<GM>(LX * VEC, p.C, p.D)));
  if (backward) k_scan_bwd<TIO, VEC, LX, GM, CONVEX, WHOLE><<<grid, kBwdThreads, 0, s>>>(p);
  else k_scan_fwd<TIO, VEC, LX, GM, CONVEX, WHOLE><<<grid, kFwdThreads, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename TIO, int VEC, int LX, int GM, bool CONVEX>
int launch_convex(const ScanParams& p, bool backward, hipStream_t s) {
  // heads of several channels are whole vectors of them
  if constexpr (VEC > 1 && GM != kScanHeadLog)
    if (p.C % VEC) return launch_whole<TIO, VEC, LX, GM, CONVEX, false>(p, backward, s);
  return launch_whole<TIO, VEC, LX, GM, CONVEX, true>(p, backward, s);
}

template <typename TIO, int VEC, int LX, int GM>
int launch_variant(const ScanParams& p, bool backward, hipStream_t s) {
  return p.convex ? launch_convex<TIO, VEC, LX, GM, true>(p, backward, s)
                  : launch_convex<TIO, VEC, LX, GM, false>(p, backward, s);
}

template <typename TIO, int GM>
int launch_gate(const ScanParams& p, bool backward, hipStream_t s) {
  constexpr int VEC = 16 / sizeof(TIO);
  if constexpr (GM == kScanHeadLog) {
    // heads wider than 128 channels need a tile that holds one
    if (p.D > 128) return launch_variant<TIO, VEC, 256 / VEC, GM>(p, backward, s);
    return launch_variant<TIO, VEC, 128 / VEC, GM>(p, backward, s);
  } else {
    // less than a vector of channels in all: one channel a lane
    if (p.C < VEC) return launch_variant<TIO, 1, 64, GM>(p, backward, s);
    return launch_variant<TIO, VEC, 128 / VEC, GM>(p, backward, s);
  }
}

template <typename TIO>
int launch_type(const ScanParams& p, bool backward, hipStream_t s) {
  switch (p.gate) {
    case kScanLog: return launch_gate<TIO, kScanLog>(p, backward, s);
    case kScanHeadLog: return launch_gate<TIO, kScanHeadLog>(p, backward, s);
    case kScanSoftplus: return launch_gate<TIO, kScanSoftplus>(p, backward, s);
    default: return launch_gate<TIO, kScanSigmoid>(p, backward, s);
  }
}

template <typename TIO, int VEC, int GM>
int launch_step_variant(const ScanStepParams& p, hipStream_t s) {
  const int64_t blocks = int64_t(p.N) * ((p.C + 256 * VEC - 1) / (256 * VEC));
  k_scan_step<TIO, VEC, GM><<<dim3(unsigned(blocks)), 256, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename TIO, int GM>
int launch_step_gate(const ScanStepParams& p, hipStream_t s) {
  constexpr int VEC = sizeof(TIO) == 2 ? 8 : 4;
  if (GM != kScanHeadLog && p.C % VEC) return launch_step_variant<TIO, 1, GM>(p, s);
  return launch_step_variant<TIO, VEC, GM>(p, s);
}

template <typename TIO>
int launch_step_type(const ScanStepParams& p, hipStream_t s) {
  switch (p.gate) {
    case kScanLog: return launch_step_gate<TIO, kScanLog>(p, s);
    case kScanHeadLog: return launch_step_gate<TIO, kScanHeadLog>(p, s);
    case kScanSoftplus: return launch_step_gate<TIO, kScanSoftplus>(p, s);
    default: return launch_step_gate<TIO, kScanSigmoid>(p, s);
  }
}

}  // namespace

int launch_scan(const ScanParams& p, bool backward, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.N == 0 || p.C == 0) return 0;
  return p.dtype == GDR_BF16 ? launch_type<bf16>(p, backward, s) : launch_type<float>(p, backward, s);
}

int launch_scan_params(const ScanParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const int hb = param_heads(p.D);
  const dim3 heads((p.H + hb - 1) / hb);
  if (p.runs) {
    k_scan_param_runs<<<dim3((p.C + 63) / 64, kParamSplit), 256, 0, s>>>(p);
    k_scan_params<double><<<heads, kParamThreads, 0, s>>>(p, p.runs, kParamSplit);
  } else {
    k_scan_params<float><<<heads, kParamThreads, 0, s>>>(p, p.part, p.NT);
  }
  return static_cast<int>(hipGetLastError());
}

int launch_scan_prologue(const ScanParams& p, int TT, const ScanBatch& b, bool clear, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const int64_t n = clear ? int64_t(p.NT) * p.C : 0;
  const int64_t blocks = std::max<int64_t>(b.n, std::min<int64_t>((n + 511) / 512, 2048));
  if (blocks == 0) return 0;
  k_scan_prologue<<<dim3(unsigned(blocks)), 256, 0, s>>>(p.counters, scan_counters(p.C), clear ? p.words : nullptr, n,
                                                         p.tab, TT, bwd_tile(p.gate, p.D > 128, p.convex), b);
  return static_cast<int>(hipGetLastError());
}

int launch_scan_step(const ScanStepParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.N == 0) return 0;
  return p.dtype == GDR_BF16 ? launch_step_type<bf16>(p, s) : launch_step_type<float>(p, s);
}

}  // namespace gdr
