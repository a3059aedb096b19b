// Gated linear recurrence s_t = a_t s_{t-1} + m_t x_t, forward and backward, and
// its single-token step.
//
// A tile is kScanTile tokens of one sequence by CT channels.  A workgroup's
// threads are LX lanes across the channels (VEC each, one 16-byte load a token)
// by LY groups along the tokens; a group's L tokens stay in registers.  The
// recurrence is affine in the state, so a group folds its tokens into
// s_out = A s_in + S, the groups are composed in order through LDS by one thread
// per channel, and each group runs its tokens again from its own starting state.
// The backward needs the states before each token and the reverse recurrence
//   ds_t = dy_t + e_{t+1},  e_t = a_t ds_t,  e_{T+1} = dht
// which folds the same way (e_out = A e_in + E with the same A), so it reads
// the inputs once and recomputes the states from the tile's starting state that
// the forward left in the workspace.
#include <hip/hip_runtime.h>

#include "gdr_device.h"
#include "gdr_gate.h"
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr int kTT = kScanTile;

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

__device__ __forceinline__ ScanTile get_tile(const ScanParams& p, int i) {
  if (p.dense_T < 0) return p.tab[i];
  const int per = max(1, (p.dense_T + kTT - 1) / kTT);
  const int b = i / per, j = i - b * per;
  return ScanTile{b * p.dense_T + j * kTT, min(kTT, p.dense_T - j * kTT), b, j};
}

// The tile's gate: log decays (and what the gradient needs) of VEC channels.
template <typename TIO, int VEC, int GM>
struct Gate {
  float eA[VEC], bias[VEC];
  __device__ __forceinline__ void init(const ScanParams& p, int c0) {
    if constexpr (GM == kScanSoftplus || GM == kScanSigmoid) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        eA[v] = expf(p.A_log[(c0 + v) / p.D]);
        bias[v] = p.dt_bias[c0 + v];
      }
    }
  }
  __device__ __forceinline__ float log_decay(float g, int v, float gs) const {
    if constexpr (GM == kScanSoftplus) return gate_log<TIO, 0>(g + bias[v], eA[v], gs);
    else if constexpr (GM == kScanSigmoid) return gate_log<TIO, 1>(g + bias[v], eA[v], gs);
    else return g;
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

template <typename TIO, int VEC, int LX, int GM>
__global__ __launch_bounds__(256) void k_scan_fwd(const ScanParams p) {
  typedef Geo<VEC, LX> G;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  __shared__ float sA[LY][CT], sS[LY][CT], sC[CT];
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int cstep = tile_channels<GM>(CT, p.D);
  const int cbase = blockIdx.x * cstep, cend = min(p.C, cbase + cstep);
  const int c0 = cbase + lx * VEC;
  const bool on = c0 < cend;
  Gate<TIO, VEC, GM> gate;
  if (on) gate.init(p, c0);

  // tiles of this sequence, in order
  const int n = blockIdx.y;
  int first = 0, count = 0;
  if (p.dense_T >= 0) {
    count = max(1, (p.dense_T + kTT - 1) / kTT);
    first = n * count;
  } else {
    // tiles are in sequence order: find this sequence's run
    int lo = 0, hi = p.NT;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.tab[mid].seq < n) lo = mid + 1; else hi = mid;
    }
    first = lo;
    count = 0;
    while (first + count < p.NT && p.tab[first + count].seq == n) ++count;
  }
  for (int c = tid; c < cend - cbase; c += 256)
    sC[c] = p.h0 ? p.h0[int64_t(n) * p.C + cbase + c] : 0.f;
  __syncthreads();
  for (int j = 0; j < count; ++j) {
    const ScanTile tile = get_tile(p, first + j);
    float a[L][VEC], u[L][VEC], A[VEC], S[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) { A[v] = 1.f; S[v] = 0.f; }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int r = ly * L + i;
      const bool live = on && r < tile.len;
      if (live) {
        const int64_t t = tile.t_start + r;
        float g[VEC], x[VEC];
        GateRaw<TIO, VEC, GM>::unpack(GateRaw<TIO, VEC, GM>::load(p, t, c0), g);
        Vec<TIO, VEC>::unpack(Vec<TIO, VEC>::load(p.x, t * p.C + c0), x);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float l = gate.log_decay(g[v], v, p.gate_scale);
          a[i][v] = exp_io<TIO>(l);
          u[i][v] = p.convex ? one_minus_exp(l, a[i][v]) * x[v] : x[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) { a[i][v] = 1.f; u[i][v] = 0.f; }
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        S[v] = a[i][v] * S[v] + u[i][v];
        A[v] *= a[i][v];
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) { sA[ly][lx * VEC + v] = A[v]; sS[ly][lx * VEC + v] = S[v]; }
    __syncthreads();
    for (int c = tid; c < cend - cbase; c += 256) {
      float s = sC[c];
      p.carry[int64_t(first + j) * p.C + cbase + c] = s;
#pragma unroll
      for (int y = 0; y < LY; ++y) {
        const float Ay = sA[y][c], Sy = sS[y][c];
        sS[y][c] = s;
        s = Ay * s + Sy;
      }
      sC[c] = s;
      if (j == count - 1 && p.ht) p.ht[int64_t(n) * p.C + cbase + c] = s;
    }
    __syncthreads();
    float s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = sS[ly][lx * VEC + v];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int r = ly * L + i;
#pragma unroll
      for (int v = 0; v < VEC; ++v) s[v] = a[i][v] * s[v] + u[i][v];
      if (on && r < tile.len) Vec<TIO, VEC>::store(p.y, (int64_t(tile.t_start) + r) * p.C + c0, s);
    }
    __syncthreads();
  }
}

template <typename TIO, int VEC, int LX, int GM>
__global__ __launch_bounds__(256) void k_scan_bwd(const ScanParams p) {
  typedef Geo<VEC, LX> G;
  constexpr int L = G::L, LY = G::LY, CT = G::CT;
  constexpr bool kPar = GM == kScanSoftplus || GM == kScanSigmoid;
  __shared__ float sA[LY][CT], sS[LY][CT], sE[LY][CT], sC[CT];
  __shared__ float sG[GM == kScanHeadLog ? kTT : 1][LX + 1];
  const int tid = threadIdx.x, lx = tid % LX, ly = tid / LX;
  const int cstep = tile_channels<GM>(CT, p.D);
  const int cbase = blockIdx.x * cstep, cend = min(p.C, cbase + cstep);
  const int c0 = cbase + lx * VEC;
  const bool on = c0 < cend;
  Gate<TIO, VEC, GM> gate;
  if (on) gate.init(p, c0);

  const int n = blockIdx.y;
  int first = 0, count = 0;
  if (p.dense_T >= 0) {
    count = max(1, (p.dense_T + kTT - 1) / kTT);
    first = n * count;
  } else {
    int lo = 0, hi = p.NT;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (p.tab[mid].seq < n) lo = mid + 1; else hi = mid;
    }
    first = lo;
    count = 0;
    while (first + count < p.NT && p.tab[first + count].seq == n) ++count;
  }
  for (int c = tid; c < cend - cbase; c += 256)
    sC[c] = p.dht ? p.dht[int64_t(n) * p.C + cbase + c] : 0.f;
  __syncthreads();
  for (int j = count - 1; j >= 0; --j) {
    const ScanTile tile = get_tile(p, first + j);
    float a[L][VEC], before[L][VEC], A[VEC], S[VEC], E[VEC];
    float g[L][VEC], x[L][VEC], dy[L][VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) { A[v] = 1.f; S[v] = 0.f; E[v] = 0.f; }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const int r = ly * L + i;
      const bool live = on && r < tile.len;
      if (live) {
        const int64_t t = tile.t_start + r;
        GateRaw<TIO, VEC, GM>::unpack(GateRaw<TIO, VEC, GM>::load(p, t, c0), g[i]);
        Vec<TIO, VEC>::unpack(Vec<TIO, VEC>::load(p.x, t * p.C + c0), x[i]);
        Vec<TIO, VEC>::unpack(Vec<TIO, VEC>::load(p.dy, t * p.C + c0), dy[i]);
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        float u = 0.f;
        if (live) {
          const float l = gate.log_decay(g[i][v], v, p.gate_scale);
          a[i][v] = exp_io<TIO>(l);
          u = p.convex ? one_minus_exp(l, a[i][v]) * x[i][v] : x[i][v];
        } else {
          a[i][v] = 1.f;
          dy[i][v] = 0.f;
          g[i][v] = 0.f;
          x[i][v] = 0.f;
        }
        S[v] = a[i][v] * S[v] + u;
        A[v] *= a[i][v];
      }
    }
#pragma unroll
    for (int i = L - 1; i >= 0; --i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) E[v] = a[i][v] * (dy[i][v] + E[v]);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sA[ly][lx * VEC + v] = A[v];
      sS[ly][lx * VEC + v] = S[v];
      sE[ly][lx * VEC + v] = E[v];
    }
    __syncthreads();
    for (int c = tid; c < cend - cbase; c += 256) {
      float s = p.carry[int64_t(first + j) * p.C + cbase + c], e = sC[c];
#pragma unroll
      for (int y = 0; y < LY; ++y) {
        const float Sy = sS[y][c];
        sS[y][c] = s;
        s = sA[y][c] * s + Sy;
      }
#pragma unroll
      for (int y = LY - 1; y >= 0; --y) {
        const float Ey = sE[y][c];
        sE[y][c] = e;
        e = sA[y][c] * e + Ey;
      }
      sC[c] = e;
      if (j == 0 && p.dh0) p.dh0[int64_t(n) * p.C + cbase + c] = e;
    }
    __syncthreads();
    float s[VEC], e[VEC], sumz[VEC], sumA[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      s[v] = sS[ly][lx * VEC + v];
      e[v] = sE[ly][lx * VEC + v];
      sumz[v] = sumA[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        before[i][v] = s[v];
        const float l = gate.log_decay(g[i][v], v, p.gate_scale);
        s[v] = a[i][v] * s[v] + (p.convex ? one_minus_exp(l, a[i][v]) * x[i][v] : x[i][v]);
      }
    }
#pragma unroll
    for (int i = L - 1; i >= 0; --i) {
      const int r = ly * L + i;
      float dx[VEC], dg[VEC];
      float dsum = 0.f;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float ds = dy[i][v] + e[v];
        e[v] = a[i][v] * ds;
        const float dl = e[v] * (p.convex ? before[i][v] - x[i][v] : before[i][v]);
        if constexpr (kPar) {
          float lam, dz, dA;
          gate_log_grad<TIO, GM == kScanSoftplus ? 0 : 1>(g[i][v] + gate.bias[v], gate.eA[v], p.gate_scale, lam, dz, dA);
          dx[v] = p.convex ? one_minus_exp(lam, a[i][v]) * ds : ds;
          dg[v] = dl * dz;
          if (r < tile.len) {
            sumz[v] += dg[v];
            sumA[v] += dl * dA;
          }
        } else {
          dx[v] = p.convex ? one_minus_exp(g[i][v], a[i][v]) * ds : ds;
          dg[v] = dl;
          dsum += dl;
        }
      }
      if (on && r < tile.len) {
        const int64_t t = tile.t_start + r;
        Vec<TIO, VEC>::store(p.dx, t * p.C + c0, dx);
        if constexpr (GM != kScanHeadLog) Vec<TIO, VEC>::store(p.dg, t * p.C + c0, dg);
      }
      if constexpr (GM == kScanHeadLog) sG[r][lx] = dsum;
    }
    if constexpr (GM == kScanHeadLog) {
      __syncthreads();
      const int heads = (cend - cbase) / p.D, lanes = p.D / VEC, h0 = cbase / p.D;
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
      for (int c = tid; c < cend - cbase; c += 256) {
        float z = 0.f, A2 = 0.f;
#pragma unroll
        for (int y = 0; y < LY; ++y) { z += sS[y][c]; A2 += sE[y][c]; }
        float* q = p.part + int64_t(first + j) * 2 * p.C + cbase + c;
        q[0] = z;
        q[p.C] = A2;
      }
    }
    __syncthreads();
  }
}

// ddt_bias and dA_log from the tiles' partial sums: a workgroup per head.
__global__ __launch_bounds__(256) void k_scan_params(const ScanParams p) {
  __shared__ double red[256];
  const int h = blockIdx.x, tid = threadIdx.x;
  double dA = 0.0;
  for (int d = 0; d < p.D; ++d) {
    double z = 0.0;
    for (int i = tid; i < p.NT; i += 256) {
      const float* q = p.part + int64_t(i) * 2 * p.C + int64_t(h) * p.D + d;
      z += q[0];
      dA += q[p.C];
    }
    red[tid] = z;
    __syncthreads();
    for (int m = 128; m; m >>= 1) {
      if (tid < m) red[tid] += red[tid + m];
      __syncthreads();
    }
    if (tid == 0) p.ddt_bias[int64_t(h) * p.D + d] = float(red[0]);
    __syncthreads();
  }
  red[tid] = dA;
  __syncthreads();
  for (int m = 128; m; m >>= 1) {
    if (tid < m) red[tid] += red[tid + m];
    __syncthreads();
  }
  if (tid == 0) p.dA_log[h] = float(red[0]);
}

__global__ __launch_bounds__(64) void k_scan_tables(ScanTile* tab, const ScanBatch b) {
  const int i = blockIdx.x;
  const int len = b.len[i], tiles = max(1, (len + kTT - 1) / kTT);
  for (int j = threadIdx.x; j < tiles; j += 64)
    tab[b.tile0[i] + j] = ScanTile{b.t_start[i] + j * kTT, min(kTT, len - j * kTT), b.seq0 + i, j};
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
  Gate<TIO, VEC, GM> gate;
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
      const float l = gate.log_decay(g[v], v, p.gate_scale);
      const float a = exp_io<TIO>(l);
      s[v] = a * s[v] + (p.convex ? one_minus_exp(l, a) * x[v] : x[v]);
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
  const dim3 grid((p.C + cstep - 1) / cstep, p.N);
  if (backward) k_scan_bwd<TIO, VEC, LX, GM><<<grid, 256, 0, s>>>(p);
  else k_scan_fwd<TIO, VEC, LX, GM><<<grid, 256, 0, s>>>(p);
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
  k_scan_params<<<dim3(p.H), 256, 0, s>>>(p);
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
