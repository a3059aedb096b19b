// The gated delta rule's single-token step on a pool of states (gdr_step).
//
//   S' = S Diag(e^lambda),  d = beta (v - S' kn),  S = S' + d kn^T,
//   o = scale S qn = scale (S' qn + d (kn . qn))
// Every row of S (one value channel) is independent given q, k and the gate, so
// eight lanes hold a row in registers, both products with the row reduce over
// those lanes alone, and the state is read and written once.  Each group of eight
// lanes forms the norms of q and k itself from its share of the channels: no LDS
// and no barrier but for the search for rows that share a slot.  The state's bytes
// bound the step: 250 rows of 32 heads, D = 128, move 1 GB in 189 us (5.5 TB/s; a
// large copy moves 4.9).  Small batches are bound by latencies that follow each other:
// the state's load is on its way during the search for shared slots, but q, k, the gate
// and v are asked for only behind its two barriers.  One row of 16 heads takes 3.4 us
// in a graph; 33 rows of 16 heads, D = 64, fp32, per-channel gate, 5.9, where the bytes
// would take 3.6.
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "gdr_gate.h"
#include "gdr_layer.h"

namespace gdr {
namespace {

// Lane j of a row's eight holds channels 32 m + 4 j .. + 3, m < D / 32: the eight
// lanes read 128 contiguous bytes of the row at a time.
template <typename TIO, int D>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int j, float (&x)[D / 8]) {
#pragma unroll
  for (int m = 0; m < D / 32; ++m) {
    float y[4];
    IO<TIO>::load4(base, off + 32 * m + 4 * j, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * m + e] = y[e];
  }
}

// R: rows of the state per workgroup (32 per pass)
template <typename TIO, int D, int GM, int R>
__global__ __launch_bounds__(256) void k_step(const StepParams p) {
  constexpr int E = D / 8, NP = R / 32, SPLIT = D / R;
  const int64_t id = blockIdx.x;
  const int part = int(id % SPLIT);
  const int h = int(id / SPLIT % p.H);
  int n = int(id / SPLIT / p.H);
  const int slot = p.slots ? p.slots[n] : n;
  if (slot < 0 || slot >= p.P) return;
  const int j = threadIdx.x & 7, row0 = part * R + (threadIdx.x >> 3);
  float* st = p.state + (int64_t(slot) * p.H + h) * (D * D);
  float S[NP][E];
#pragma unroll
  for (int i = 0; i < NP; ++i) load_row<float, D>(st, int64_t(row0 + 32 * i) * D, j, S[i]);
  // the state is on its way; meanwhile: the row is another's if an earlier one names
  // the slot, and takes the later ones that do along
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
  for (;;) {
    const int64_t hk = int64_t(n) * p.Hk + h / p.G, hv = int64_t(n) * p.H + h;
    float q[E], k[E], a[E], qq = 0.f, kk = 0.f, kq = 0.f;
    load_row<TIO, D>(p.q, hk * D, j, q);
    load_row<TIO, D>(p.k, hk * D, j, k);
    if constexpr (GM == 0) {
      a[0] = fast_exp2(IO<TIO>::load1(p.g, hv) * kLog2e);
#pragma unroll
      for (int e = 1; e < E; ++e) a[e] = a[0];
    } else {
      const float eA = expf(p.A_log[h]);
      float bias[E];
      load_row<TIO, D>(p.g, hv * D, j, a);
      load_row<float, D>(p.dt_bias, int64_t(h) * D, j, bias);
#pragma unroll
      for (int e = 0; e < E; ++e)
        a[e] = fast_exp2(gate_log2<GM - 1>(fmaf(a[e], kLog2e, bias[e] * kLog2e), eA, p.gate_scale));
    }
    const float beta = 1.f / (1.f + fast_exp2(-kLog2e * IO<TIO>::load1(p.b, hv)));
#pragma unroll
    for (int e = 0; e < E; ++e) {
      qq += q[e] * q[e];
      kk += k[e] * k[e];
    }
    const float rq = rsqrtf(group_sum_dpp<8>(qq) + 1e-6f), rk = rsqrtf(group_sum_dpp<8>(kk) + 1e-6f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] *= rq;
      k[e] *= rk;
      kq += k[e] * q[e];
    }
    kq = group_sum_dpp<8>(kq);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = row0 + 32 * i;
      float r = 0.f, o = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        S[i][e] *= a[e];
        r += S[i][e] * k[e];
        o += S[i][e] * q[e];
      }
      r = group_sum_dpp<8>(r);
      o = group_sum_dpp<8>(o);
      const float d = beta * (IO<TIO>::load1(p.v, hv * D + row) - r);
#pragma unroll
      for (int e = 0; e < E; ++e) S[i][e] += d * k[e];
      if (j == 0) IO<TIO>::store1(p.o, hv * D + row, p.scale * (o + d * kq));
    }
    if (!later) break;
    do ++n; while (n < p.N && p.slots[n] != slot);
    if (n >= p.N) break;
  }
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int m = 0; m < D / 32; ++m)
      IO<float>::store4(st, int64_t(row0 + 32 * i) * D + 32 * m + 4 * j, S[i][4 * m], S[i][4 * m + 1], S[i][4 * m + 2],
                        S[i][4 * m + 3]);
}

// Rows of the state per workgroup: 32 with one decay per head, 64 with per-channel
// gates, whose functions every eight lanes work out again.  In us, in a graph:
//                                        per head        per channel
//                                        32      64       32      64
//   250 rows, 32 heads of 128, bf16     192     207      218     195
//   250 rows, 32 heads of 64, bf16       50      52       61      54
//   33 rows, 16 heads of 64, fp32       5.5     5.3      6.7     5.9
//   8 rows, 16 heads of 128, bf16       5.0     5.1      6.1     5.9
//   1 row, 16 heads of 128, bf16        3.4     3.8      4.2     4.6
// A single row with a per-channel gate loses 0.4 us by 64, a small fp32 batch with one
// decay per head 0.2 by 32: neither is given a rule of its own.
template <typename TIO, int D, int GM>
int launch_gate(const StepParams& p, hipStream_t s) {
  constexpr int R = GM == 0 ? 32 : 64;
  k_step<TIO, D, GM, R><<<dim3(unsigned(int64_t(p.N) * p.H * (D / R))), 256, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename TIO, int D>
int launch_dim(const StepParams& p, hipStream_t s) {
  if (p.gate == 0) return launch_gate<TIO, D, 0>(p, s);
  return p.gate_fn == 0 ? launch_gate<TIO, D, 1>(p, s) : launch_gate<TIO, D, 2>(p, s);
}

}  // namespace

int launch_step(const StepParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (p.N == 0) return 0;
  if (p.dtype == GDR_BF16) return p.D == 128 ? launch_dim<bf16, 128>(p, s) : launch_dim<bf16, 64>(p, s);
  return p.D == 128 ? launch_dim<float, 128>(p, s) : launch_dim<float, 64>(p, s);
}

}  // namespace gdr
