// Host side of the operators around the delta rule (see gdr.h): argument checks,
// the recurrence's workspace and tile table, and the launch sequences.  Nothing
// here allocates or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "gdr_check.h"
#include "gdr_layer.h"

namespace {

using namespace gdr::check;
using gdr::set_error;

// ---------------------------------------------------------------------------
// gated linear recurrence
// ---------------------------------------------------------------------------

int64_t tiles_of(int64_t len, int64_t tile) { return std::max<int64_t>(1, (len + tile - 1) / tile); }

int scan_gate(const gdr_scan_shape* s) {
  if (s->gate == GDR_GATE_CHANNEL) return gdr::kScanSoftplus;
  if (s->gate == GDR_GATE_CHANNEL_SIGMOID) return gdr::kScanSigmoid;
  return s->D == 1 ? gdr::kScanLog : gdr::kScanHeadLog;
}


// NT_out: backward tiles over all sequences (there are no more forward tiles).
gdr_status check_scan_shape(const gdr_scan_shape* s, int64_t* NT_out) {
  if (!s) return set_error(GDR_EINVAL, "shape is NULL");
  if (s->gate != GDR_GATE_SCALAR && s->gate != GDR_GATE_CHANNEL && s->gate != GDR_GATE_CHANNEL_SIGMOID)
    return set_error(GDR_EINVAL, "unknown gate %d", s->gate);
  if (s->gate == GDR_GATE_CHANNEL_SIGMOID && !(s->gate_scale <= 0.f && s->gate_scale > -1e30f))
    return set_error(GDR_EINVAL, "gate_scale %g must be finite and <= 0 (a log decay)", double(s->gate_scale));
  if (s->dtype != GDR_BF16 && s->dtype != GDR_F32) return set_error(GDR_EINVAL, "unknown dtype %d", s->dtype);
  if (s->convex != 0 && s->convex != 1) return set_error(GDR_EINVAL, "convex %d must be 0 or 1", s->convex);
  if (s->H < 1 || s->B < 1 || s->T < 0 || s->N < 0 || s->D < 1) return set_error(GDR_EINVAL, "bad B/T/H/D/N");
  if (s->D > 256 || (s->D != 1 && s->D % 8 != 0))
    return set_error(GDR_EUNSUPPORTED, "head dim %d must be 1 or a multiple of 8 up to 256", s->D);
  int64_t NT = 0;
  const int tile = gdr::bwd_tile(scan_gate(s), s->D > 128, s->convex);
  if (s->cu_seqlens_host == nullptr) {
    if (s->N != s->B) return set_error(GDR_EINVAL, "dense shape needs N == B (N=%d, B=%d)", s->N, s->B);
    NT = int64_t(s->B) * tiles_of(s->T, tile);
  } else {
    if (s->B != 1) return set_error(GDR_EINVAL, "varlen shape needs B == 1");
    if (s->N < 1) return set_error(GDR_EINVAL, "varlen shape needs N >= 1");
    const int64_t* cu = s->cu_seqlens_host;
    if (cu[0] != 0) return set_error(GDR_EINVAL, "cu_seqlens[0] = %lld, expected 0", (long long)cu[0]);
    for (int n = 0; n < s->N; ++n) {
      if (cu[n + 1] < cu[n]) return set_error(GDR_EINVAL, "cu_seqlens decreases at %d", n);
      if (cu[n + 1] > s->T) return set_error(GDR_EINVAL, "cu_seqlens[%d] = %lld > T = %d", n + 1, (long long)cu[n + 1], s->T);
      NT += tiles_of(cu[n + 1] - cu[n], tile);
    }
    if (cu[s->N] != s->T) return set_error(GDR_EINVAL, "cu_seqlens[N] = %lld != T = %d", (long long)cu[s->N], s->T);
  }
  const int64_t C = int64_t(s->H) * s->D, tokens = int64_t(s->B) * s->T;
  if (C > (int64_t(1) << 21) || tokens >= (int64_t(1) << 31) || tokens * C >= (int64_t(1) << 40) ||
      NT * ((C + 63) / 64) * 256 >= gdr::kMaxThreads)
    return set_error(GDR_EUNSUPPORTED, "problem too large for one launch and 32-bit tile indexing");
  *NT_out = NT;
  return GDR_OK;
}

struct ScanLayout {
  size_t tab = 0, counters = 0, words = 0, carry = 0, part = 0, runs = 0, total = 0;
};

ScanLayout scan_layout(const gdr_scan_shape* s, int64_t NT) {
  ScanLayout L;
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off = align256(off + bytes); return o; };
  const size_t C = size_t(s->H) * s->D;
  L.tab = take(s->cu_seqlens_host ? NT * sizeof(gdr::ScanTile) : 0);
  L.counters = take(size_t(gdr::scan_counters(int(C))) * gdr::kScanCounterStep * 4);
  L.words = take((NT * C + 1) * 8);
  L.carry = take(NT * C * 4);
  L.part = take(s->gate != GDR_GATE_SCALAR ? NT * 2 * C * 4 : 0);
  L.runs = take(s->gate != GDR_GATE_SCALAR && NT >= gdr::kParamSplitTiles ? gdr::kParamSplit * 2 * C * 8 : 0);
  L.total = off;
  return L;
}

gdr_status check_scan_inputs(const gdr_scan_shape* s, const gdr_scan_inputs* in, bool tokens) {
  if (!in) return set_error(GDR_EINVAL, "inputs is NULL");
  const bool par = s->gate != GDR_GATE_SCALAR;
  if (!par && (in->A_log || in->dt_bias)) return set_error(GDR_EINVAL, "scalar gate takes no A_log/dt_bias");
  if (par && (!in->A_log || !in->dt_bias)) return set_error(GDR_EINVAL, "per-channel gate needs A_log and dt_bias");
  const Arg a[] = {{in->x, "input x", tokens}, {in->g, "input g", tokens}, {in->A_log, "A_log", false},
                   {in->dt_bias, "dt_bias", false}, {in->h0, "h0", false}};
  return check_ptrs(a, 5);
}

int64_t fwd_tiles(const gdr_scan_shape* s) {
  if (!s->cu_seqlens_host) return int64_t(s->B) * tiles_of(s->T, gdr::fwd_tile(scan_gate(s), s->D > 128));
  int64_t n = 0;
  for (int i = 0; i < s->N; ++i) n += tiles_of(s->cu_seqlens_host[i + 1] - s->cu_seqlens_host[i], gdr::fwd_tile(scan_gate(s), s->D > 128));
  return n;
}

// NT: the direction's tiles.
gdr::ScanParams scan_params(const gdr_scan_shape* s, const gdr_scan_inputs* in, int64_t NT, const ScanLayout& L,
                            void* ws) {
  gdr::ScanParams p;
  std::memset(&p, 0, sizeof(p));
  p.H = s->H; p.D = s->D; p.C = s->H * s->D; p.N = s->N;
  p.gate = scan_gate(s); p.dtype = s->dtype; p.convex = s->convex; p.gate_scale = s->gate_scale;
  p.NT = int32_t(NT);
  p.dense_T = s->cu_seqlens_host ? -1 : s->T;
  p.x = in->x; p.g = in->g; p.A_log = in->A_log; p.dt_bias = in->dt_bias; p.h0 = in->h0;
  char* w = static_cast<char*>(ws);
  p.tab = reinterpret_cast<gdr::ScanTile*>(w + L.tab);
  // as many tiles as sequences: none waits for another
  p.words = NT > s->N ? reinterpret_cast<uint64_t*>(w + L.words) : nullptr;
  p.counters = reinterpret_cast<uint32_t*>(w + L.counters);
  p.carry = reinterpret_cast<float*>(w + L.carry);
  p.part = reinterpret_cast<float*>(w + L.part);
  p.runs = NT >= gdr::kParamSplitTiles ? reinterpret_cast<double*>(w + L.runs) : nullptr;
  return p;
}

// What a call's main kernel finds: the words cleared where tiles wait for others, and
// the tile table of a packed problem (sequences by value, kScanBatch a launch).
gdr_status scan_prologue(const gdr_scan_shape* s, const gdr::ScanParams& p, int tile, void* stream) {
  gdr::ScanBatch b;
  std::memset(&b, 0, sizeof(b));
  bool clear = p.words != nullptr;
  if (!s->cu_seqlens_host)
    return clear ? hip_status(gdr::launch_scan_prologue(p, tile, b, true, stream), "scan prologue kernel") : GDR_OK;
  const int saved_tile = gdr::bwd_tile(p.gate, p.D > 128, p.convex);
  int64_t row = 0, saved = 0;
  for (int n0 = 0; n0 < s->N; n0 += gdr::kScanBatch) {
    b.n = std::min(gdr::kScanBatch, s->N - n0);
    b.seq0 = n0;
    for (int i = 0; i < b.n; ++i) {
      const int64_t start = s->cu_seqlens_host[n0 + i], len = s->cu_seqlens_host[n0 + i + 1] - start;
      b.t_start[i] = int32_t(start);
      b.len[i] = int32_t(len);
      b.tile0[i] = int32_t(row);
      b.saved0[i] = int32_t(saved);
      row += tiles_of(len, tile);
      saved += tiles_of(len, saved_tile);
    }
    const gdr_status st = hip_status(gdr::launch_scan_prologue(p, tile, b, clear, stream), "scan prologue kernel");
    if (st != GDR_OK) return st;
    clear = false;
  }
  return GDR_OK;
}

// ---------------------------------------------------------------------------
// norm
// ---------------------------------------------------------------------------

gdr_status check_norm_shape(const gdr_norm_shape* s) {
  if (!s) return set_error(GDR_EINVAL, "shape is NULL");
  if (s->dtype != GDR_BF16 && s->dtype != GDR_F32) return set_error(GDR_EINVAL, "unknown dtype %d", s->dtype);
  if (s->rows < 0 || s->width < 1) return set_error(GDR_EINVAL, "bad rows/width");
  if (!(s->eps >= 0.f && s->eps < 1e30f)) return set_error(GDR_EINVAL, "eps %g must be finite and >= 0", double(s->eps));
  if (s->width > gdr::kNormMaxWidth)
    return set_error(GDR_EUNSUPPORTED, "width %d above %d", s->width, gdr::kNormMaxWidth);
  if (s->rows >= (int64_t(1) << 31) ||
      gdr::norm_fwd_blocks(s->rows, s->width, s->dtype) * gdr::norm_fwd_threads(s->width, s->dtype) >= gdr::kMaxThreads)
    return set_error(GDR_EUNSUPPORTED, "too many rows (%lld of width %d) for one launch", (long long)s->rows, s->width);
  return GDR_OK;
}

gdr_status norm_forward(const gdr_norm_shape* s, const void* x, const void* res, const float* w, void* y, void* q,
                        float* scales, void* res_out, void* stream) {
  const bool rows = s->rows > 0;
  if (rows && (res == nullptr) != (res_out == nullptr))
    return set_error(GDR_EINVAL, "res and res_out go together");
  const Arg a[] = {{x, "x", rows}, {res, "res", false}, {w, "w", false}, {res_out, "res_out", false}};
  const gdr_status st = check_ptrs(a, 4);
  if (st != GDR_OK) return st;
  if (y && y == res_out) return set_error(GDR_EINVAL, "y and res_out are the same tensor");
  gdr::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = s->rows; p.width = s->width; p.dtype = s->dtype; p.eps = s->eps; p.group = s->group;
  p.x = x; p.res = res; p.w = w; p.y = y; p.q = q; p.scales = scales; p.res_out = res_out;
  return hip_status(gdr::launch_norm(p, stream), "norm kernel");
}

size_t norm_ws(const gdr_norm_shape* s) {
  return align256(size_t(gdr::norm_bwd_partials(s->rows, s->width, s->dtype)) * size_t(s->width) * 4);
}

}  // namespace

extern "C" {

gdr_status gdr_scan_workspace_bytes(const gdr_scan_shape* shape, size_t* bytes) {
  int64_t NT = 0;
  const gdr_status st = check_scan_shape(shape, &NT);
  if (st != GDR_OK) return st;
  if (!bytes) return set_error(GDR_EINVAL, "bytes is NULL");
  *bytes = scan_layout(shape, NT).total;
  return GDR_OK;
}

gdr_status gdr_scan_fwd(const gdr_scan_shape* shape, const gdr_scan_inputs* in, void* ws, size_t ws_bytes, void* y,
                        float* ht, void* stream) {
  int64_t NT = 0;
  gdr_status st = check_scan_shape(shape, &NT);
  if (st != GDR_OK) return st;
  const bool tokens = int64_t(shape->B) * shape->T > 0;
  if ((st = check_scan_inputs(shape, in, tokens)) != GDR_OK) return st;
  const Arg a[] = {{y, "y", tokens}, {ht, "ht", false}};
  if ((st = check_ptrs(a, 2)) != GDR_OK) return st;
  const ScanLayout L = scan_layout(shape, NT);
  if ((st = check_ws(L.total, ws, ws_bytes)) != GDR_OK) return st;
  gdr::ScanParams p = scan_params(shape, in, fwd_tiles(shape), L, ws);
  p.y = y;
  p.ht = ht;
  if ((st = scan_prologue(shape, p, gdr::fwd_tile(p.gate, p.D > 128), stream)) != GDR_OK) return st;
  return hip_status(gdr::launch_scan(p, false, stream), "scan kernel");
}

gdr_status gdr_scan_bwd(const gdr_scan_shape* shape, const gdr_scan_inputs* in, const void* dy, const float* dht,
                        void* ws, size_t ws_bytes, const gdr_scan_grads* grads, void* stream) {
  int64_t NT = 0;
  gdr_status st = check_scan_shape(shape, &NT);
  if (st != GDR_OK) return st;
  const bool tokens = int64_t(shape->B) * shape->T > 0;
  if ((st = check_scan_inputs(shape, in, tokens)) != GDR_OK) return st;
  if (!grads) return set_error(GDR_EINVAL, "grads is NULL");
  const bool par = shape->gate != GDR_GATE_SCALAR;
  if (!par && (grads->dA_log || grads->ddt_bias))
    return set_error(GDR_EINVAL, "scalar gate has no dA_log/ddt_bias outputs");
  const Arg a[] = {{dy, "dy", tokens}, {dht, "dht", false}, {grads->dx, "output dx", tokens},
                   {grads->dg, "output dg", tokens}, {grads->dh0, "dh0", false}, {grads->dA_log, "dA_log", par},
                   {grads->ddt_bias, "ddt_bias", par}};
  if ((st = check_ptrs(a, 7)) != GDR_OK) return st;
  const ScanLayout L = scan_layout(shape, NT);
  if ((st = check_ws(L.total, ws, ws_bytes)) != GDR_OK) return st;
  gdr::ScanParams p = scan_params(shape, in, NT, L, ws);
  p.dy = dy; p.dht = dht;
  p.dx = grads->dx; p.dg = grads->dg; p.dh0 = grads->dh0; p.dA_log = grads->dA_log; p.ddt_bias = grads->ddt_bias;
  if ((st = scan_prologue(shape, p, gdr::bwd_tile(p.gate, p.D > 128, p.convex), stream)) != GDR_OK) return st;
  if ((st = hip_status(gdr::launch_scan(p, true, stream), "scan gradient kernel")) != GDR_OK) return st;
  return par ? hip_status(gdr::launch_scan_params(p, stream), "parameter reduction kernel") : GDR_OK;
}

gdr_status gdr_scan_step(const gdr_scan_shape* shape, const gdr_scan_inputs* in, float* state, int32_t P,
                         const int32_t* slots, void* y, void* stream) {
  int64_t NT = 0;
  gdr_status st = check_scan_shape(shape, &NT);
  if (st != GDR_OK) return st;
  if (shape->cu_seqlens_host || shape->T != 1) return set_error(GDR_EINVAL, "a step takes a dense shape with T == 1");
  if ((st = check_scan_inputs(shape, in, true)) != GDR_OK) return st;
  if (in->h0) return set_error(GDR_EINVAL, "a step takes its states from the pool, not from h0");
  if ((st = check_pool(shape->N, state, P, slots)) != GDR_OK) return st;
  const Arg a[] = {{y, "y", true}};
  if ((st = check_ptrs(a, 1)) != GDR_OK) return st;
  gdr::ScanStepParams p;
  std::memset(&p, 0, sizeof(p));
  p.H = shape->H; p.D = shape->D; p.C = shape->H * shape->D; p.N = shape->N; p.P = P;
  p.gate = scan_gate(shape); p.dtype = shape->dtype; p.convex = shape->convex; p.gate_scale = shape->gate_scale;
  p.x = in->x; p.g = in->g; p.A_log = in->A_log; p.dt_bias = in->dt_bias;
  p.slots = slots; p.state = state; p.y = y;
  return hip_status(gdr::launch_scan_step(p, stream), "scan step kernel");
}

gdr_status gdr_step(const gdr_shape* shape, const gdr_inputs* in, float* state, int32_t P, const int32_t* slots,
                    void* o, void* stream) {
  size_t bytes = 0;
  gdr_shape unsplit;
  if (shape) {
    unsplit = *shape;
    unsplit.seq_split = 1;   // there is no sequence to split, whatever the shape says
  }
  // checks the shape; a step needs no workspace
  gdr_status st = gdr_workspace_bytes(shape ? &unsplit : nullptr, &bytes);
  if (st != GDR_OK) return st;
  if (shape->cu_seqlens_host || shape->T != 1) return set_error(GDR_EINVAL, "a step takes a dense shape with T == 1");
  if (int64_t(shape->N) * shape->H * (shape->Dk / 32) * 256 >= gdr::kMaxThreads)
    return set_error(GDR_EUNSUPPORTED, "too many rows (%d of %d heads) for one launch", shape->N, shape->H);
  if (!in) return set_error(GDR_EINVAL, "inputs is NULL");
  const bool par = shape->gate != GDR_GATE_SCALAR;
  if (!par && (in->A_log || in->dt_bias)) return set_error(GDR_EINVAL, "scalar gate takes no A_log/dt_bias");
  if (par && (!in->A_log || !in->dt_bias)) return set_error(GDR_EINVAL, "per-channel gate needs A_log and dt_bias");
  if (in->h0) return set_error(GDR_EINVAL, "a step takes its states from the pool, not from h0");
  const Arg a[] = {{in->q, "input q", true}, {in->k, "input k", true}, {in->v, "input v", true}, {in->g, "input g", true},
                   {in->beta_logit, "input beta_logit", true}, {in->A_log, "A_log", false},
                   {in->dt_bias, "dt_bias", false}, {o, "o", true}};
  if ((st = check_ptrs(a, 8)) != GDR_OK) return st;
  if ((st = check_pool(shape->N, state, P, slots)) != GDR_OK) return st;
  gdr::StepParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = shape->N; p.H = shape->H; p.D = shape->Dk; p.P = P;
  p.Hk = shape->Hk > 0 ? shape->Hk : shape->H;
  p.G = p.H / p.Hk;
  p.gate = par ? 1 : 0;
  p.gate_fn = shape->gate == GDR_GATE_CHANNEL_SIGMOID ? 1 : 0;
  p.dtype = shape->dtype; p.scale = shape->scale; p.gate_scale = shape->gate_scale;
  p.q = in->q; p.k = in->k; p.v = in->v; p.g = in->g; p.b = in->beta_logit;
  p.A_log = in->A_log; p.dt_bias = in->dt_bias;
  p.slots = slots; p.state = state; p.o = o;
  return hip_status(gdr::launch_step(p, stream), "step kernel");
}

gdr_status gdr_norm_fwd(const gdr_norm_shape* shape, const void* x, const void* res, const float* w, void* y,
                        void* res_out, void* stream) {
  const gdr_status st = check_norm_shape(shape);
  if (st != GDR_OK) return st;
  const Arg a[] = {{y, "y", shape->rows > 0}};
  const gdr_status sp = check_ptrs(a, 1);
  if (sp != GDR_OK) return sp;
  return norm_forward(shape, x, res, w, y, nullptr, nullptr, res_out, stream);
}

gdr_status gdr_norm_quant(const gdr_norm_shape* shape, const void* x, const void* res, const float* w, void* q,
                          float* scales, void* res_out, void* stream) {
  const gdr_status st = check_norm_shape(shape);
  if (st != GDR_OK) return st;
  if (shape->group != 0 && shape->group != 128)
    return set_error(GDR_EUNSUPPORTED, "group %d not in {0, 128}", shape->group);
  const Arg a[] = {{q, "q", shape->rows > 0}, {scales, "scales", shape->rows > 0}};
  const gdr_status sp = check_ptrs(a, 2);
  if (sp != GDR_OK) return sp;
  return norm_forward(shape, x, res, w, nullptr, q, scales, res_out, stream);
}

gdr_status gdr_norm_workspace_bytes(const gdr_norm_shape* shape, size_t* bytes) {
  const gdr_status st = check_norm_shape(shape);
  if (st != GDR_OK) return st;
  if (!bytes) return set_error(GDR_EINVAL, "bytes is NULL");
  *bytes = norm_ws(shape);
  return GDR_OK;
}

gdr_status gdr_norm_bwd(const gdr_norm_shape* shape, const void* r, const float* w, const void* dy, const void* dres,
                        void* ws, size_t ws_bytes, void* dx, float* dw, void* stream) {
  gdr_status st = check_norm_shape(shape);
  if (st != GDR_OK) return st;
  const bool rows = shape->rows > 0;
  const Arg a[] = {{r, "r", rows}, {w, "w", false}, {dy, "dy", rows}, {dres, "dres", false}, {dx, "dx", rows},
                   {dw, "dw", false}};
  if ((st = check_ptrs(a, 6)) != GDR_OK) return st;
  if (dw && (st = check_ws(norm_ws(shape), ws, ws_bytes)) != GDR_OK) return st;
  gdr::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = shape->rows; p.width = shape->width; p.dtype = shape->dtype; p.eps = shape->eps;
  p.x = r; p.w = w; p.dy = dy; p.dres = dres; p.dx = dx; p.dw = dw;
  p.part = dw ? static_cast<float*>(ws) : nullptr;
  return hip_status(gdr::launch_norm_bwd(p, stream), "norm gradient kernel");
}

}  // extern "C"
