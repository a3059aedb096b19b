// Host side of linear attention with a decay for each head (see gdr.h): argument checks,
// the split of sequences into segments, the workspace and the launch sequences.  Nothing
// here allocates or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "gdr_check.h"
#include "gdr_layer.h"
#include "gdr_lin.h"

namespace {

using namespace gdr::check;
using gdr::set_error;

int64_t parts_of(int64_t len, int64_t part) { return std::max<int64_t>(1, (len + part - 1) / part); }

int64_t seq_start(const gdr_lin_shape* s, int n) { return s->cu_seqlens_host ? s->cu_seqlens_host[n] : int64_t(n) * s->T; }
int64_t seq_len(const gdr_lin_shape* s, int n) {
  return s->cu_seqlens_host ? s->cu_seqlens_host[n + 1] - s->cu_seqlens_host[n] : s->T;
}

gdr_status check_lin_shape(const gdr_lin_shape* s) {
  if (!s) return set_error(GDR_EINVAL, "shape is NULL");
  if (s->dtype != GDR_BF16 && s->dtype != GDR_F32) return set_error(GDR_EINVAL, "unknown dtype %d", s->dtype);
  if (s->H < 1 || s->B < 1 || s->T < 0 || s->N < 0 || s->D < 1) return set_error(GDR_EINVAL, "bad B/T/H/D/N");
  if (s->D != 64 && s->D != 128) return set_error(GDR_EUNSUPPORTED, "head dim %d not in {64, 128}", s->D);
  if (s->Hk < 0 || (s->Hk > 0 && s->H % s->Hk != 0))
    return set_error(GDR_EINVAL, "Hk %d must be 0 or divide H %d", s->Hk, s->H);
  if (!(s->scale > -1e30f && s->scale < 1e30f)) return set_error(GDR_EINVAL, "scale %g must be finite", double(s->scale));
  if (s->cu_seqlens_host == nullptr) {
    if (s->N != s->B) return set_error(GDR_EINVAL, "dense shape needs N == B (N=%d, B=%d)", s->N, s->B);
  } else {
    if (s->B != 1) return set_error(GDR_EINVAL, "varlen shape needs B == 1");
    if (s->N < 1) return set_error(GDR_EINVAL, "varlen shape needs N >= 1");
    const int64_t* cu = s->cu_seqlens_host;
    if (cu[0] != 0) return set_error(GDR_EINVAL, "cu_seqlens[0] = %lld, expected 0", (long long)cu[0]);
    for (int n = 0; n < s->N; ++n) {
      if (cu[n + 1] < cu[n]) return set_error(GDR_EINVAL, "cu_seqlens decreases at %d", n);
      if (cu[n + 1] > s->T) return set_error(GDR_EINVAL, "cu_seqlens[%d] = %lld > T = %d", n + 1, (long long)cu[n + 1], s->T);
    }
    if (cu[s->N] != s->T) return set_error(GDR_EINVAL, "cu_seqlens[N] = %lld != T = %d", (long long)cu[s->N], s->T);
  }
  // at most 16 workgroups of 256 threads for every state or block, and the bytes of a block's
  // rows within 32 bits
  constexpr int64_t most = gdr::kMaxThreads / (16 * 256);
  const int64_t blocks = int64_t(s->B) * s->T / gdr::kLinBlock + s->N;
  if (s->H > (1 << 16) || blocks >= most || blocks * s->H >= most)
    return set_error(GDR_EUNSUPPORTED, "problem too large for one launch and 32-bit indexing");
  return GDR_OK;
}

// Tokens per segment: whole blocks, as many as a model of the time finds best.  In units of a
// block's turn in one of the four output kernels (4.2 to 4.8 us at T = 32768, 16 heads of 128,
// bf16, with every compute unit at work): segments run one to a compute unit, split ones' own
// states cost a quarter more, and the states between them 3 and another 3 for each 256.
// Segments of one length take whole rounds of the compute units; of a pack's, which are not,
// half a segment is lost at the end.  Measured, forward and backward together, heads of 128,
// bf16, in us for segments of
//                          1 block     2     4     8    16    32
//   T = 512, 4 heads            51      61    87    90 (no split)
//   T = 2048, 4 heads           64      69    93   145
//   T = 2048, 16 heads         135      98   102   151
//   4 x 1000, 8 heads          134      96   100   149
//   T = 8192, 16 heads                        245   216
//   T = 32768, 16 heads                                   697   677
//   4 x 4095, 32 heads                                    675   667
// and, heads of 64, T = 8192, 8 heads: 85 for 2, 74 for 4, 90 for 8; 12 uneven sequences, 32
// heads: 1830 for 66, 1681 for 33, 1661 for 22.
// Neither the type nor D is in the model.  fp32, heads of 128, us: T = 16384, 16 heads, 916 for
// 16 (the model's), 966 for 8; T = 4096, 16 heads, 274 for 4 (the model's), 324 for 2; 4 x 4095,
// 32 heads, 1758 for 32 (the model's), 1811 for 16.  Off the best: fp32, T = 2048, 4 heads, 123
// for 2 (the model's), 92 for 1; 32 heads of 64, T = 16384, 348 for 32 (the model's), 324 for 16,
// and fp32 680 and 601.
int64_t segment_of(const gdr_lin_shape* s) {
  constexpr int64_t kUnits = 256;
  int64_t blocks = 0, longest = 0;
  const bool pack = s->cu_seqlens_host != nullptr;
  for (int n = 0; n < (pack ? s->N : 1); ++n) {
    const int64_t b = parts_of(seq_len(s, n), gdr::kLinBlock);
    blocks += b;
    longest = std::max(longest, b);
  }
  if (!pack) blocks *= s->N;
  int64_t best = longest, least = INT64_MAX;
  for (int64_t k = 1; k <= std::min<int64_t>(longest, 1024); k += std::max<int64_t>(1, k / 8)) {
    const int64_t seg = parts_of(longest, k);
    const int64_t groups = (pack ? blocks / seg + s->N / 2 : s->N * parts_of(longest, seg)) * s->H;
    const int64_t turns = pack ? std::max(seg, blocks * s->H / kUnits + seg / 2) : parts_of(groups, kUnits) * seg;
    const int64_t time = k == 1 ? 4 * turns : 5 * turns + 12 + 12 * groups / kUnits;
    if (time < least) {
      least = time;
      best = seg;
    }
  }
  return best * gdr::kLinBlock;
}

struct LinLayout {
  int64_t seg = 0, NC = 0;
  bool split = false;
  size_t tab = 0, row0 = 0, st = 0, dst = 0, part = 0, total = 0;
};

LinLayout lin_layout(const gdr_lin_shape* s, bool backward) {
  LinLayout L;
  L.seg = segment_of(s);
  if (s->cu_seqlens_host) {
    for (int n = 0; n < s->N; ++n) {
      const int64_t k = parts_of(seq_len(s, n), L.seg);
      L.NC += k;
      L.split |= k > 1;
    }
  } else {
    const int64_t k = parts_of(s->T, L.seg);
    L.NC = k * s->N;
    L.split = k > 1;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
  L.tab = take(s->cu_seqlens_host ? L.NC * sizeof(gdr::LinSeg) : 0);
  L.row0 = take(s->cu_seqlens_host ? (size_t(s->N) + 1) * 4 : 0);
  const size_t states = L.split ? size_t(L.NC) * s->H * s->D * s->D * 4 : 0;
  L.st = take(states);
  L.dst = take(backward ? states : 0);
  const bool grouped = s->Hk > 0 && s->Hk < s->H;
  L.part = take(backward && grouped ? size_t(s->B) * s->T * s->H * s->D * 4 : 0);
  L.total = off;
  return L;
}

gdr_status check_lin_inputs(const gdr_lin_inputs* in, bool tokens) {
  if (!in) return set_error(GDR_EINVAL, "inputs is NULL");
  const Arg a[] = {{in->q, "input q", tokens}, {in->k, "input k", tokens}, {in->v, "input v", tokens},
                   {in->log_decay, "log_decay", true}, {in->h0, "h0", false}};
  return check_ptrs(a, 5);
}

gdr::LinParams lin_params(const gdr_lin_shape* s, const gdr_lin_inputs* in, const LinLayout& L, void* ws) {
  gdr::LinParams p;
  std::memset(&p, 0, sizeof(p));
  p.H = s->H; p.Hk = s->Hk > 0 ? s->Hk : s->H; p.G = p.H / p.Hk;
  p.D = s->D; p.N = s->N; p.T = s->B * s->T;
  p.NC = int32_t(L.NC); p.seg = int32_t(L.seg);
  p.dense_T = s->cu_seqlens_host ? -1 : s->T;
  p.dense_nseg = s->cu_seqlens_host ? 0 : int32_t(parts_of(s->T, L.seg));
  p.dtype = s->dtype; p.split = L.split; p.scale = s->scale;
  p.q = in->q; p.k = in->k; p.v = in->v; p.log_decay = in->log_decay; p.h0 = in->h0;
  char* w = static_cast<char*>(ws);
  p.tab = reinterpret_cast<gdr::LinSeg*>(w + L.tab);
  p.row0 = reinterpret_cast<int32_t*>(w + L.row0);
  p.st = reinterpret_cast<float*>(w + L.st);
  p.dst = reinterpret_cast<float*>(w + L.dst);
  p.part = reinterpret_cast<float*>(w + L.part);
  return p;
}

// The segments of a packed problem, its sequences by value, kLinBatch a launch.
gdr_status lin_table(const gdr_lin_shape* s, const gdr::LinParams& p, void* stream) {
  if (!s->cu_seqlens_host) return GDR_OK;
  gdr::LinBatch b;
  std::memset(&b, 0, sizeof(b));
  int64_t row = 0;
  for (int n0 = 0; n0 < s->N; n0 += gdr::kLinBatch) {
    b.n = std::min(gdr::kLinBatch, s->N - n0);
    b.seq0 = n0;
    for (int i = 0; i < b.n; ++i) {
      b.t0[i] = int32_t(seq_start(s, n0 + i));
      b.len[i] = int32_t(seq_len(s, n0 + i));
      b.row0[i] = int32_t(row);
      row += parts_of(b.len[i], p.seg);
    }
    const gdr_status st = hip_status(gdr::launch_lin_table(p, b, stream), "segment table kernel");
    if (st != GDR_OK) return st;
  }
  return GDR_OK;
}

}  // namespace

extern "C" {

gdr_status gdr_lin_workspace_bytes(const gdr_lin_shape* shape, int32_t backward, size_t* bytes) {
  const gdr_status st = check_lin_shape(shape);
  if (st != GDR_OK) return st;
  if (!bytes) return set_error(GDR_EINVAL, "bytes is NULL");
  *bytes = lin_layout(shape, backward != 0).total;
  return GDR_OK;
}

gdr_status gdr_lin_fwd(const gdr_lin_shape* shape, const gdr_lin_inputs* in, void* ws, size_t ws_bytes, void* o,
                       float* ht, void* stream) {
  gdr_status st = check_lin_shape(shape);
  if (st != GDR_OK) return st;
  const bool tokens = int64_t(shape->B) * shape->T > 0;
  if ((st = check_lin_inputs(in, tokens)) != GDR_OK) return st;
  const Arg a[] = {{o, "o", tokens}, {ht, "ht", false}};
  if ((st = check_ptrs(a, 2)) != GDR_OK) return st;
  const LinLayout L = lin_layout(shape, false);
  if ((st = check_ws(L.total, ws, ws_bytes)) != GDR_OK) return st;
  gdr::LinParams p = lin_params(shape, in, L, ws);
  p.o = o;
  p.ht = ht;
  if ((st = lin_table(shape, p, stream)) != GDR_OK) return st;
  if ((st = hip_status(gdr::launch_lin_states(p, false, stream), "segment state kernels")) != GDR_OK) return st;
  return hip_status(gdr::launch_lin_fwd(p, stream), "linear attention kernel");
}

gdr_status gdr_lin_bwd(const gdr_lin_shape* shape, const gdr_lin_inputs* in, const void* dO, const float* dht,
                       void* ws, size_t ws_bytes, const gdr_lin_grads* grads, void* stream) {
  gdr_status st = check_lin_shape(shape);
  if (st != GDR_OK) return st;
  const bool tokens = int64_t(shape->B) * shape->T > 0;
  if ((st = check_lin_inputs(in, tokens)) != GDR_OK) return st;
  if (!grads) return set_error(GDR_EINVAL, "grads is NULL");
  const Arg a[] = {{dO, "dO", tokens}, {dht, "dht", false}, {grads->dq, "output dq", tokens},
                   {grads->dk, "output dk", tokens}, {grads->dv, "output dv", tokens}, {grads->dh0, "dh0", false}};
  if ((st = check_ptrs(a, 6)) != GDR_OK) return st;
  const LinLayout L = lin_layout(shape, true);
  if ((st = check_ws(L.total, ws, ws_bytes)) != GDR_OK) return st;
  gdr::LinParams p = lin_params(shape, in, L, ws);
  p.dO = dO; p.dht = dht;
  p.dq = grads->dq; p.dk = grads->dk; p.dv = grads->dv; p.dh0 = grads->dh0;
  if ((st = hip_status(gdr::launch_lin_states(p, true, stream), "segment state gradient kernels")) != GDR_OK) return st;
  return hip_status(gdr::launch_lin_bwd(p, stream), "linear attention gradient kernels");
}

gdr_status gdr_lin_step(const gdr_lin_shape* shape, const gdr_lin_inputs* in, float* state, int32_t P,
                        const int32_t* slots, void* o, void* stream) {
  gdr_status st = check_lin_shape(shape);
  if (st != GDR_OK) return st;
  if (shape->cu_seqlens_host || shape->T != 1) return set_error(GDR_EINVAL, "a step takes a dense shape with T == 1");
  if ((st = check_lin_inputs(in, true)) != GDR_OK) return st;
  if (in->h0) return set_error(GDR_EINVAL, "a step takes its states from the pool, not from h0");
  const Arg a[] = {{o, "o", true}};
  if ((st = check_ptrs(a, 1)) != GDR_OK) return st;
  if ((st = check_pool(shape->N, state, P, slots)) != GDR_OK) return st;
  gdr::LinStepParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = shape->N; p.H = shape->H; p.Hk = shape->Hk > 0 ? shape->Hk : shape->H; p.G = p.H / p.Hk;
  p.D = shape->D; p.P = P; p.dtype = shape->dtype; p.scale = shape->scale;
  p.q = in->q; p.k = in->k; p.v = in->v; p.log_decay = in->log_decay;
  p.slots = slots; p.state = state; p.o = o;
  return hip_status(gdr::launch_lin_step(p, stream), "linear attention step kernel");
}

}  // extern "C"
