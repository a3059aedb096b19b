// Internal declarations of the operators around the delta rule: the gated linear
// recurrence (gdr_scan.hip), the row norm (gdr_norm.hip) and the delta rule's
// single-token step (gdr_step.hip).  Their argument checks are in gdr_layer.cpp.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../../include/gdr.h"

namespace gdr {

// Threads of a launch: a launch of as many is refused by the runtime, so the shape
// checks refuse it before anything is enqueued.
constexpr int64_t kMaxThreads = int64_t(1) << 32;

// How the recurrence's kernels read the gate.
enum ScanGate {
  kScanLog = 0,       // one log decay per channel (scalar gate, D = 1)
  kScanHeadLog = 1,   // one log decay per head (scalar gate, D > 1)
  kScanSoftplus = 2,
  kScanSigmoid = 3,
};

// Tokens per tile of the recurrence, backward and forward.  A decay per head is one
// register a token, which leaves room for longer tiles, unless the head is so wide
// (over 128 channels) that a tile holds twice the channels; plain decays per channel
// take a longer tile in the backward, but not in its convex form, which would spill 160
// to 220 registers.  The convex forms are at the 256-register limit: with a decay per
// head they spill 2 (bf16) or 26 to 30 (fp32, backward), with the sigmoid gate 17 to 39
// in the backward, and are faster so than in shorter tiles.  Forward, backward in us at
// T = 32768 (bf16) or 16384 (fp32):
//   32 heads of 128, decay per head      256, 128 tokens   128, 64
//     bf16, convex                           130, 205      141, 253
//     bf16                                   123, 202      138, 247
//     fp32, convex                           127, 186      126, 189
//     fp32                                   114, 168      113, 177
//   4096 channels, backward                 128 tokens        64
//     bf16                                     278           318
//     fp32                                     252           258
//     bf16, convex                             803           352
//     fp32, convex                             494           260
//   sigmoid, convex, bf16, backward          64 tokens        32
//     16 heads of 128                          254           266
//     2051 channels                            371           359
constexpr bool scan_long(int gate, bool wide) { return gate == kScanHeadLog && !wide; }
constexpr int bwd_tile(int gate, bool wide, bool convex) {
  return scan_long(gate, wide) || (gate == kScanLog && !convex) ? 128 : 64;
}
constexpr int fwd_tile(int gate, bool wide) { return scan_long(gate, wide) ? 256 : 128; }
// Tiles of a sequence of `len` tokens, at least one.  Unsigned: len + tile - 1 may pass
// 2^31.  (len - 1) / tile + 1 cost the convex form with a decay per head two more spilled
// registers (T = 32768, 32 heads of 128, forward: 133 us for 130).
constexpr int scan_tiles(int len, int tile) {
  const int n = int((uint32_t(len) + uint32_t(tile) - 1) / uint32_t(tile));
  return n > 1 ? n : 1;
}

// One row per tile: at most a tile's tokens of one sequence.  A sequence without
// tokens has one empty tile, so that its states are passed through.
struct ScanTile {
  int32_t t_start, len, seq;
  int32_t idx, after;   // tiles of the sequence before and after it
  int32_t saved;        // its (first) backward tile: the row of the saved states
};

// Sequences handed to the table kernel by value, kScanBatch per launch.
constexpr int kScanBatch = 120;
struct ScanBatch {
  int32_t n, seq0, pad[2];
  int32_t t_start[kScanBatch], len[kScanBatch], tile0[kScanBatch], saved0[kScanBatch];
};
static_assert(sizeof(ScanBatch) <= 2048, "kernel argument size");

// Counters of the tiles taken, one per channel tile and each in a cache line of its
// own: one counter for all of them bounds a launch (13 ns a workgroup, 210 us for the
// 16384 tiles of T = 32768 and 4096 channels).
constexpr int kScanCounterStep = 32;
inline int scan_counters(int C) { return C / 64 + 1; }   // channel tiles: 64 channels or more each

// Runs in which the backward's per-tile parameter sums are added up, from this many
// tiles on.
constexpr int kParamSplit = 16, kParamSplitTiles = 128;

struct ScanParams {
  int32_t H, D, C, N;          // C = H D channels
  int32_t gate, dtype, convex;
  int32_t NT;                  // this direction's tiles over all sequences
  int32_t dense_T;             // dense: tokens per sequence; -1: the tiles are in `tab`
  float gate_scale;
  const void *x, *g, *dy;
  const float *A_log, *dt_bias, *h0, *dht;
  void *y, *dx, *dg;
  float *ht, *dh0, *dA_log, *ddt_bias;
  ScanTile* tab;
  float* carry;                // [backward tiles][C] state at the start of each
  uint64_t* words;             // [NT][C] published folds and states; NULL: every sequence is one tile
  uint32_t* counters;          // tiles taken, per channel tile (kScanCounterStep apart)
  float* part;                 // [NT][2][C] partial sums of ddt_bias and dA_log
  double* runs;                // [kParamSplit][2][C] sums of runs of tiles; NULL: few tiles
};

// The tile rows of a batch (of TT tokens) and, with `clear`, the counters and words.
int launch_scan_prologue(const ScanParams& p, int TT, const ScanBatch& b, bool clear, void* stream);
int launch_scan(const ScanParams& p, bool backward, void* stream);
int launch_scan_params(const ScanParams& p, void* stream);

struct ScanStepParams {
  int32_t H, D, C, N, P;
  int32_t gate, dtype, convex;
  float gate_scale;
  const void *x, *g;
  const float *A_log, *dt_bias;
  const int32_t* slots;
  float* state;
  void* y;
};
int launch_scan_step(const ScanStepParams& p, void* stream);

constexpr int kNormMaxWidth = 32768;
constexpr int kNormPartials = 512;   // workgroups of the backward, each with a row of partial sums of dw

struct NormParams {
  int64_t rows;
  int32_t width, dtype, group;
  float eps;
  const void *x, *res, *dy, *dres;
  const float* w;
  void *y, *res_out, *q, *dx;
  float *scales, *dw, *part;
};
int launch_norm(const NormParams& p, void* stream);        // y, or q and scales
int launch_norm_bwd(const NormParams& p, void* stream);
int norm_bwd_partials(int64_t rows, int32_t width, int32_t dtype);
int64_t norm_fwd_blocks(int64_t rows, int32_t width, int32_t dtype);
int norm_fwd_threads(int32_t width, int32_t dtype);   // of a workgroup

struct StepParams {
  int32_t N, H, Hk, G, D, P;
  int32_t gate, gate_fn, dtype;   // gate: 0 per head, 1 per channel; gate_fn as in Params
  float scale, gate_scale;
  const void *q, *k, *v, *g, *b;
  const float *A_log, *dt_bias;
  const int32_t* slots;
  float* state;
  void* o;
};
int launch_step(const StepParams& p, void* stream);

}  // namespace gdr
