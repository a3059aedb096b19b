// Internal declarations of linear attention with a decay for each head: gdr_lin.cpp
// (checks, workspace, launch sequences) and gdr_lin.hip (kernels).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../../include/gdr.h"

namespace gdr {

constexpr int kLinBlock = 64;   // tokens per block: one turn of the kernels' loops

// A segment: a run of whole blocks of one sequence that one workgroup walks through
// with the state in registers (the last block of a sequence may be partial).
struct LinSeg {
  int32_t t0, len, seq;
  int32_t idx, nseg;   // its place among the sequence's segments
};

// Sequences handed to the table kernel by value, kLinBatch per launch.
constexpr int kLinBatch = 120;
struct LinBatch {
  int32_t n, seq0, pad[2];
  int32_t t0[kLinBatch], len[kLinBatch], row0[kLinBatch];
};
static_assert(sizeof(LinBatch) <= 2048, "kernel argument size");

struct LinParams {
  int32_t H, Hk, G, D, N, T;   // T: tokens over all sequences
  int32_t NC;                  // segments (chunk_head_at's name for them)
  int32_t seg;                 // tokens per segment
  int32_t dense_T, dense_nseg; // dense: tokens and segments per sequence; dense_T < 0: the segments are in `tab`
  int32_t dtype;
  int32_t split;               // some sequence has several segments
  float scale;
  const void *q, *k, *v, *dO;
  const float *log_decay, *h0, *dht;
  void *o, *dq, *dk, *dv;
  float *ht, *dh0;
  LinSeg* tab;
  int32_t* row0;               // [N + 1] first segment of each sequence, packed problems
  float *st, *dst;             // [NC][H][D][D]: the state a segment starts from, forward and backward
  float* part;                 // grouped heads: dq or dk per value head, [T][H][D]
};

int launch_lin_table(const LinParams& p, const LinBatch& b, void* stream);
// States of the segments and their composition; `backward`: of the state's gradient.
int launch_lin_states(const LinParams& p, bool backward, void* stream);
int launch_lin_fwd(const LinParams& p, void* stream);
int launch_lin_bwd(const LinParams& p, void* stream);

struct LinStepParams {
  int32_t N, H, Hk, G, D, P, dtype;
  float scale;
  const void *q, *k, *v;
  const float* log_decay;
  const int32_t* slots;
  float* state;
  void* o;
};
int launch_lin_step(const LinStepParams& p, void* stream);

}  // namespace gdr
