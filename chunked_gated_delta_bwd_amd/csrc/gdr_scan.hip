// Gated linear recurrence s_t = a_t s_{t-1} + m_t x_t, forward and backward, and
// its single-token step.
//
// A tile is kScanTile tokens of one sequence by CT channels, a workgroup's work.
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
// Between tiles: every tile publishes its fold (A, S) and, once it knows the state
// it starts from, the state it ends with.  A tile looks back over its predecessors,
// composing folds, until it meets a published end state; so the inputs cross HBM
// once and no tile waits for a chain of others to finish.  A value and its tag are
// one 64-bit word, stored and loaded as one atomic access at device scope, so no
// fence is needed.  Workgroups take tiles in an order (by a counter) in which a
// tile's predecessors were taken before it: they are running or done, and publish
// their folds without waiting for anybody, so every wait ends.  (Waits are
// bounded all the same: should the workspace be overwritten by someone else during
// the call, the states become NaN and the kernel ends.)
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gdr_device.h"
#include "gdr_gate.h"
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kTT = kScanTile;

// ---- published words ----
enum : uint32_t { kTagNone = 0, kTagFold = 1, kTagState = 2 };
constexpr int kMaxPolls = 1 << 20;

__device__ __forceinline__ void put(uint64_t* w, float v, uint32_t tag) {
  __hip_atomic_store(w, (uint64_t(tag) << 32) | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get(const uint64_t* w) {
  return __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t tag_of(uint64_t w) { return uint32_t(w >> 32); }
__device__ __forceinline__ float val_of(uint64_t w) { return __uint_as_float(uint32_t(w)); }

// The state that reaches a tile of one channel from the tiles `step` rows apart
// before it (`w` addresses the nearest one's words: A at w, S at w + C), `count` of
// them up to the sequence's first, which always publishes a state.
__device__ __forceinline__ float look_back(const uint64_t* w, int64_t step, int C, int count) {
  constexpr int kAhead = 4;   // predecessors whose words are loaded at a time
  float A = 1.f, S = 0.f;
  int polls = 0;
  for (int k = 0; k < count; k += kAhead) {
    uint64_t wa[kAhead], ws[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t o = -step * min(k + i, count - 1);
      ws[i] = get(w + o + C);
      wa[i] = get(w + o);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t o = -step * min(k + i, count - 1);
      while (tag_of(ws[i]) == kTagNone || (tag_of(ws[i]) == kTagFold && tag_of(wa[i]) == kTagNone)) {
        if (++polls > kMaxPolls) return __builtin_nanf("");
        ws[i] = get(w + o + C);
        wa[i] = get(w + o);
      }
      S += A * val_of(ws[i]);
      if (tag_of(ws[i]) == kTagState) return S;
      A *= val_of(wa[i]);
    }
  }
  return S;
}

// VEC consecutive elements: one vector access for VEC > 1
template <typename TIO, int VEC>
struct Vec {
  typedef typename IO<TIO>::Raw8 Raw;
  static __device__ __forceinline__ Raw load(const void* b, int64_t o) { return IO<TIO>::load_raw8(b, o); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[VEC]) { IO<TIO>::unpack8(r, x); }
  static __device__ __forceinline__ void store(void* b, int64_t o, const float (&x)[VEC]) { IO<TIO>::store8(b, o, x); }
};
template <typename TIO>
struct Vec<TIO, 4> {
  typedef typename IO<TIO>::Raw4 Raw;
  static __device__ __forceinline__ Raw load(const void* b, int64_t o) { return IO<TIO>::load_raw4(b, o); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[4]) { IO<TIO>::unpack4(r, x); }
  static __device__ __forceinline__ void store(void* b, int64_t o, const float (&x)[4]) {
    IO<TIO>::store4(b, o, x[0], x[1], x[2], x[3]);
  }
};
template <typename TIO>
struct Vec<TIO, 1> {
  typedef float Raw;
  static __device__ __forceinline__ Raw load(const void* b, int64_t o) { return IO<TIO>::load1(b, o); }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[1]) { x[0] = r; }
  static __device__ __forceinline__ void store(void* b, int64_t o, const float (&x)[1]) { IO<TIO>::store1(b, o, x[0]); }
};

// Geometry of a variant.
template <int VEC, int LX>
struct Geo {
  static constexpr int LY = 256 / LX;
  static constexpr int L = kTT / LY;      // tokens per thread
  static constexpr int CT = LX * VEC;     // channels per tile
};

// Channels a tile advances by: CT, or with one gate per head the whole heads that
// fit (the head's gate gradient is summed inside the workgroup).
template <int GM>
__host__ __device__ __forceinline__ int tile_channels(int CT, int D) {
  return GM == kScanHeadLog ? CT / D * D : CT;
}

// The place of a tile (its row of the published words and of the saved states) in
// the order in which the workgroups take them, and the tile.
__device__ __forceinline__ ScanTile tile_at(const ScanParams& p, int order, bool backward, int& row) {
  if (p.dense_T < 0) {
    row = backward ? p.NT - 1 - order : order;
    return p.tab[row];
  }
  // all sequences' first tiles, then all second ones, ...
  const int per = max(1, (p.dense_T + kTT - 1) / kTT);
  const int level = order / p.N, seq = order - level * p.N, idx = backward ? per - 1 - level : level;
  row = seq * per + idx;
  return ScanTile{seq * p.dense_T + idx * kTT, min(kTT, p.dense_T - idx * kTT), seq, idx, per - 1 - idx};
}

// The workgroup's place in the order: its number where no tile waits for another,
// else the next of the counter.
__device__ __forceinline__ int take_order(const ScanParams& p, int* slot) {
  if (!p.words) return blockIdx.x;
  if (threadIdx.x == 0) *slot = int(atomicAdd(p.counter, 1u));
  __syncthreads();
  return *slot;
}

// The gate of VEC channels: base-2 log decays, and what its gradient needs.
template <int VEC, int GM>
struct Gate {
  float eA[VEC], bias[VEC];
  __device__ __forceinline__ void init(const ScanParams& p, int c0) {
    if constexpr (GM == kScanSoftplus || GM == kScanSigmoid) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        eA[v] = expf(p.A_log[(c0 + v) / p.D]);
        bias[v] = p.dt_bias[c0 + v] * kLog2e;
      }
    }
  }
  __device__ __forceinline__ float log2_decay(float g, int v, float gs) const {
    if constexpr (GM == kScanSoftplus) return gate_log2<0>(fmaf(g, kLog2e, bias[v]), eA[v], gs);
    else if constexpr (GM == kScanSigmoid) return gate_log2<1>(fmaf(g, kLog2e, bias[v]), eA[v], gs);
    else return g * kLog2e;
  }
};

// Raw gate values of one token: VEC of them, or the head's one.
template <typename TIO, int VEC, int GM>
struct GateRaw {
  typedef typename Vec<TIO, VEC>::Raw Raw;
  static __device__ __forceinline__ Raw load(const ScanParams& p, int64_t t, int c0) {
    return Vec<TIO, VEC>::load(p.g, t * p.C + c0);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&g)[VEC]) { Vec<TIO, VEC>::unpack(r, g); }
};
template <typename TIO, int VEC>
struct GateRaw<TIO, VEC, kScanHeadLog> {
  typedef float Raw;
  static __device__ __forceinline__ Raw load(const ScanParams& p, int64_t t, int c0) {
    return IO<TIO>::load1(p.g, t * p.H + c0 / p.D);
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&g)[VEC]) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) g[v] = r;
  }
};

// Tokens and channels of a thread, with the loads kept in bounds: rows past the
// tile's end and lanes past its channels load a valid neighbour's values, which
// are then left out (a = 1, no input).
template <typename TIO, int VEC, int LX, int GM>
__global__ __launch_bounds__(256) void k_scan_fwd(const ScanParams p) {
  typedef Geo<VEC, LX> G;
  typedef Vec<TIO, VEC> V;
  typedef GateRaw<TIO, VEC, GM> GR;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  __shared__ float sA[LY][CT], sS[LY][CT];
  __shared__ int slot;
  const int order = take_order(p, &slot);
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int cstep = tile_channels<GM>(CT, p.D);
  const int nct = (p.C + cstep - 1) / cstep;
  const int cbase = order % nct * cstep, nc = min(p.C - cbase, cstep);
  int row;
  const ScanTile tile = tile_at(p, order / nct, false, row);
  const bool on = lx * VEC < nc;
  const int c0 = cbase + (on ? lx * VEC : 0);
  float a[L][VEC], u[L][VEC];
  if (tile.len > 0) {
    typename GR::Raw rg[L];
    typename V::Raw rx[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int64_t t = int64_t(tile.t_start) + min(ly * L + i, tile.len - 1);
      rg[i] = GR::load(p, t, c0);
      rx[i] = V::load(p.x, t * p.C + c0);
    }
    Gate<VEC, GM> gate;
    gate.init(p, c0);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float g[VEC], x[VEC];
      GR::unpack(rg[i], g);
      V::unpack(rx[i], x);
      const bool live = ly * L + i < tile.len;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float l = gate.log2_decay(g[v], v, p.gate_scale);
        const float d = fast_exp2(l);
        const float w = p.convex ? one_minus_exp2(l, d) * x[v] : x[v];
        a[i][v] = live ? d : 1.f;
        u[i][v] = live ? w : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) { a[i][v] = 1.f; u[i][v] = 0.f; }
  }
  float A[VEC], S[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) { A[v] = a[0][v]; S[v] = u[0][v]; }
#pragma unroll
  for (int i = 1; i < L; ++i)
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      S[v] = fmaf(a[i][v], S[v], u[i][v]);
      A[v] *= a[i][v];
    }
#pragma unroll
  for (int v = 0; v < VEC; ++v) { sA[ly][lx * VEC + v] = A[v]; sS[ly][lx * VEC + v] = S[v]; }
  __syncthreads();
  for (int c = tid; c < nc; c += 256) {
    uint64_t* w = p.words + int64_t(row) * 2 * p.C + cbase + c;
    float s;
    if (tile.idx == 0) {
      s = p.h0 ? p.h0[int64_t(tile.seq) * p.C + cbase + c] : 0.f;
    } else {
      float At = 1.f, St = 0.f;
#pragma unroll
      for (int y = 0; y < LY; ++y) {
        St = fmaf(sA[y][c], St, sS[y][c]);
        At *= sA[y][c];
      }
      if (tile.after > 0) {
        put(w, At, kTagFold);
        put(w + p.C, St, kTagFold);
      }
      s = look_back(w - 2 * int64_t(p.C), 2 * int64_t(p.C), p.C, tile.idx);
    }
    p.carry[int64_t(row) * p.C + cbase + c] = s;
#pragma unroll
    for (int y = 0; y < LY; ++y) {
      const float Sy = sS[y][c];
      sS[y][c] = s;
      s = fmaf(sA[y][c], s, Sy);
    }
    if (tile.after > 0) put(w + p.C, s, kTagState);
    else if (p.ht) p.ht[int64_t(tile.seq) * p.C + cbase + c] = s;
  }
  __syncthreads();
  float s[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) s[v] = sS[ly][lx * VEC + v];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int r = ly * L + i;
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = fmaf(a[i][v], s[v], u[i][v]);
    if (on && r < tile.len) V::store(p.y, (int64_t(tile.t_start) + r) * p.C + c0, s);
  }
}

template <typename TIO, int VEC, int LX, int GM>
__global__ __launch_bounds__(256) void k_scan_bwd(const ScanParams p) {
  typedef Geo<VEC, LX> G;
  typedef Vec<TIO, VEC> V;
  typedef GateRaw<TIO, VEC, GM> GR;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  constexpr bool kPar = GM == kScanSoftplus || GM == kScanSigmoid;
  __shared__ float sA[LY][CT], sS[LY][CT], sE[LY][CT];
  __shared__ float sG[GM == kScanHeadLog ? kTT : 1][LX + 1];
  __shared__ int slot;
  const int order = take_order(p, &slot);
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int cstep = tile_channels<GM>(CT, p.D);
  const int nct = (p.C + cstep - 1) / cstep;
  const int cbase = order % nct * cstep, nc = min(p.C - cbase, cstep);
  int row;
  const ScanTile tile = tile_at(p, order / nct, true, row);
  const bool on = lx * VEC < nc;
  const int c0 = cbase + (on ? lx * VEC : 0);
  // per token: the decay, its base-2 logarithm, the gate's slopes (per-channel
  // gates), the input; `u` becomes the state before the token
  float a[L][VEC], l[L][VEC], dz[kPar ? L : 1][VEC], dA[kPar ? L : 1][VEC], u[L][VEC];
  typename V::Raw rx[L], rdy[L];
  if (tile.len > 0) {
    typename GR::Raw rg[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int64_t t = int64_t(tile.t_start) + min(ly * L + i, tile.len - 1);
      rg[i] = GR::load(p, t, c0);
      rx[i] = V::load(p.x, t * p.C + c0);
      rdy[i] = V::load(p.dy, t * p.C + c0);
    }
    Gate<VEC, GM> gate;
    gate.init(p, c0);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float g[VEC], x[VEC];
      GR::unpack(rg[i], g);
      V::unpack(rx[i], x);
      const bool live = ly * L + i < tile.len;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float l2;
        if constexpr (kPar) {
          gate_log2_grad<GM == kScanSoftplus ? 0 : 1>(fmaf(g[v], kLog2e, gate.bias[v]), gate.eA[v], p.gate_scale, l2,
                                                       dz[i][v], dA[i][v]);
        } else {
          l2 = g[v] * kLog2e;
        }
        const float d = fast_exp2(l2);
        const float w = p.convex ? one_minus_exp2(l2, d) * x[v] : x[v];
        l[i][v] = l2;
        a[i][v] = live ? d : 1.f;
        u[i][v] = live ? w : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        a[i][v] = 1.f;
        u[i][v] = l[i][v] = 0.f;
        if constexpr (kPar) dz[i][v] = dA[i][v] = 0.f;
      }
  }
  {
    float A[VEC], S[VEC], E[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) { A[v] = a[0][v]; S[v] = u[0][v]; E[v] = 0.f; }
#pragma unroll
    for (int i = 1; i < L; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[v] = fmaf(a[i][v], S[v], u[i][v]);
        A[v] *= a[i][v];
      }
    if (tile.len > 0) {
#pragma unroll
      for (int i = L - 1; i >= 0; --i) {
        float dy[VEC];
        V::unpack(rdy[i], dy);
        const bool live = ly * L + i < tile.len;
#pragma unroll
        for (int v = 0; v < VEC; ++v) E[v] = a[i][v] * ((live ? dy[v] : 0.f) + E[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sA[ly][lx * VEC + v] = A[v];
      sS[ly][lx * VEC + v] = S[v];
      sE[ly][lx * VEC + v] = E[v];
    }
  }
  __syncthreads();
  for (int c = tid; c < nc; c += 256) {
    uint64_t* w = p.words + int64_t(row) * 2 * p.C + cbase + c;
    float s = p.carry[int64_t(row) * p.C + cbase + c], e;
    if (tile.after == 0) {
      e = p.dht ? p.dht[int64_t(tile.seq) * p.C + cbase + c] : 0.f;
    } else {
      float At = 1.f, Et = 0.f;
#pragma unroll
      for (int y = LY - 1; y >= 0; --y) {
        Et = fmaf(sA[y][c], Et, sE[y][c]);
        At *= sA[y][c];
      }
      if (tile.idx > 0) {
        put(w, At, kTagFold);
        put(w + p.C, Et, kTagFold);
      }
      e = look_back(w + 2 * int64_t(p.C), -2 * int64_t(p.C), p.C, tile.after);
    }
#pragma unroll
    for (int y = LY - 1; y >= 0; --y) {
      const float Ey = sE[y][c];
      sE[y][c] = e;
      e = fmaf(sA[y][c], e, Ey);
    }
    if (tile.idx > 0) put(w + p.C, e, kTagState);
    else if (p.dh0) p.dh0[int64_t(tile.seq) * p.C + cbase + c] = e;
#pragma unroll
    for (int y = 0; y < LY; ++y) {
      const float Sy = sS[y][c];
      sS[y][c] = s;
      s = fmaf(sA[y][c], s, Sy);
    }
  }
  __syncthreads();
  float e[VEC], sumz[VEC], sumA[VEC];
  {
    float s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      s[v] = sS[ly][lx * VEC + v];
      e[v] = sE[ly][lx * VEC + v];
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
  if (tile.len > 0) {
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
      const int r = ly * L + i;
      const bool live = r < tile.len;
      float dx[VEC], dg[VEC], x[VEC], dy[VEC];
      V::unpack(rx[i], x);
      V::unpack(rdy[i], dy);
      float dsum = 0.f;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float ds = (live ? dy[v] : 0.f) + e[v];
        e[v] = a[i][v] * ds;
        const float dl = live ? e[v] * (p.convex ? u[i][v] - x[v] : u[i][v]) : 0.f;
        dx[v] = p.convex ? one_minus_exp2(l[i][v], a[i][v]) * ds : ds;
        if constexpr (kPar) {
          dg[v] = dl * dz[i][v];
          sumz[v] += dg[v];
          sumA[v] = fmaf(dl, dA[i][v], sumA[v]);
        } else {
          dg[v] = dl;
          dsum += dl;
        }
      }
      if (on && live) {
        const int64_t t = int64_t(tile.t_start) + r;
        V::store(p.dx, t * p.C + c0, dx);
        if constexpr (GM != kScanHeadLog) V::store(p.dg, t * p.C + c0, dg);
      }
      if constexpr (GM == kScanHeadLog) sG[r][lx] = dsum;
    }
  }
  if constexpr (GM == kScanHeadLog) {
    __syncthreads();
    const int heads = nc / p.D, lanes = p.D / VEC, h0 = cbase / p.D;
    for (int i = tid; i < tile.len * heads; i += 256) {
      const int r = i / heads, h = i - r * heads;
      float d = 0.f;
      for (int m = 0; m < lanes; ++m) d += sG[r][h * lanes + m];
      IO<TIO>::store1(p.dg, (int64_t(tile.t_start) + r) * p.H + h0 + h, d);
    }
  }
  if constexpr (kPar) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < VEC; ++v) { sS[ly][lx * VEC + v] = sumz[v]; sE[ly][lx * VEC + v] = sumA[v]; }
    __syncthreads();
    for (int c = tid; c < nc; c += 256) {
      float z = 0.f, zA = 0.f;
#pragma unroll
      for (int y = 0; y < LY; ++y) { z += sS[y][c]; zA += sE[y][c]; }
      float* q = p.part + int64_t(row) * 2 * p.C + cbase + c;
      q[0] = z;
      q[p.C] = zA;
    }
  }
}

// ddt_bias and dA_log from the tiles' partial sums: a workgroup per head (several
// narrow ones), its threads a row group each of the tiles; 64-bit sums in a fixed
// order.
constexpr int kParamThreads = 1024;
__host__ __device__ __forceinline__ int param_heads(int D) { return D >= 64 ? 1 : 64 / D; }

__global__ __launch_bounds__(kParamThreads) void k_scan_params(const ScanParams p) {
  __shared__ double sz[kParamThreads], sa[kParamThreads];
  const int h0 = blockIdx.x * param_heads(p.D), heads = min(param_heads(p.D), p.H - h0);
  const int cw = heads * p.D, groups = kParamThreads / cw;
  const int tid = threadIdx.x, c = tid % cw, g = tid / cw;
  double z = 0.0, zA = 0.0;
  if (g < groups) {
    const float* q = p.part + int64_t(h0) * p.D + c;
#pragma unroll 8
    for (int i = g; i < p.NT; i += groups) {
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

// The tile rows of up to kScanBatch sequences.
__global__ __launch_bounds__(64) void k_scan_tables(ScanTile* tab, const ScanBatch b) {
  const int i = blockIdx.x;
  const int len = b.len[i], tiles = max(1, (len + kTT - 1) / kTT);
  for (int j = threadIdx.x; j < tiles; j += 64)
    tab[b.tile0[i] + j] = ScanTile{b.t_start[i] + j * kTT, min(kTT, len - j * kTT), b.seq0 + i, j, tiles - 1 - j};
}

// Clears the counter and the published words' tags.
__global__ __launch_bounds__(256) void k_scan_clear(uint32_t* counter, uint4* words, int64_t n) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256)
    words[i] = make_uint4(0, 0, 0, 0);
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
    GateRaw<TIO, VEC, GM>::unpack(GateRaw<TIO, VEC, GM>::load(q, n, c0), g);
    Vec<TIO, VEC>::unpack(Vec<TIO, VEC>::load(p.x, int64_t(n) * p.C + c0), x);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float l = gate.log2_decay(g[v], v, p.gate_scale);
      const float a = fast_exp2(l);
      s[v] = a * s[v] + (p.convex ? one_minus_exp2(l, a) * x[v] : x[v]);
    }
    Vec<TIO, VEC>::store(p.y, int64_t(n) * p.C + c0, s);
    if (!later) break;
    do ++n; while (n < p.N && p.slots[n] != slot);
    if (n >= p.N) break;
  }
  if constexpr (VEC == 1) st[0] = s[0];
  else if constexpr (VEC == 4) IO<float>::store4(st, 0, s[0], s[1], s[2], s[3]);
  else IO<float>::store8(st, 0, s);
}

template <typename TIO, int VEC, int LX, int GM>
int launch_variant(const ScanParams& p, bool backward, hipStream_t s) {
  const int cstep = tile_channels<GM>(LX * VEC, p.D);
  const int64_t blocks = int64_t(p.NT) * ((p.C + cstep - 1) / cstep);
  if (backward) k_scan_bwd<TIO, VEC, LX, GM><<<dim3(unsigned(blocks)), 256, 0, s>>>(p);
  else k_scan_fwd<TIO, VEC, LX, GM><<<dim3(unsigned(blocks)), 256, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

// Vectors of 16 bytes where every row starts on one; one channel a lane otherwise
// (only D = 1 layers with an odd channel count).
template <typename TIO, int GM>
int launch_gate(const ScanParams& p, bool backward, hipStream_t s) {
  constexpr int VEC = sizeof(TIO) == 2 ? 8 : 4;
  if constexpr (GM == kScanHeadLog) {
    if (p.D > 128) return launch_variant<TIO, VEC, 256 / VEC, GM>(p, backward, s);
    return launch_variant<TIO, VEC, 128 / VEC, GM>(p, backward, s);
  } else {
    if (p.C % VEC) return launch_variant<TIO, 1, 64, GM>(p, backward, s);
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
  k_scan_params<<<dim3((p.H + hb - 1) / hb), kParamThreads, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

int launch_scan_clear(const ScanParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const int64_t n = int64_t(p.NT) * p.C;   // 16 bytes of words per tile and channel
  k_scan_clear<<<dim3(unsigned(std::min<int64_t>((n + 255) / 256, 2048))), 256, 0, s>>>(
      p.counter, reinterpret_cast<uint4*>(p.words), n);
  return static_cast<int>(hipGetLastError());
}

int launch_scan_tables(const ScanParams& p, const ScanBatch& b, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (b.n <= 0) return 0;
  k_scan_tables<<<dim3(b.n), 64, 0, s>>>(p.tab, b);
  return static_cast<int>(hipGetLastError());
}

int launch_scan_step(const ScanStepParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.N == 0) return 0;
  return p.dtype == GDR_BF16 ? launch_step_type<bf16>(p, s) : launch_step_type<float>(p, s);
}

}  // namespace gdr
