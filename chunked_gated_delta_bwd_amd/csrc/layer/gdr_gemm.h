// Internal declarations of the e4m3 product with scales for each 128 of the contraction
// and of the quantisation that makes its operands: gdr_gemm.cpp (checks, plan, launch
// sequences), gdr_gemm.hip and gdr_quant.hip (kernels).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../../include/gdr.h"

namespace gdr {

constexpr int kGroup = 128;   // elements of the contraction per scale

struct QuantParams {
  int64_t rows, cols;         // of x
  int32_t dtype, block, transpose;
  const void* x;
  void* q;
  float* scales;
};
int launch_quant(const QuantParams& p, void* stream);

// How a product is cut into workgroups.
struct GemmPlan {
  int32_t kind;               // 0: few rows of a; 1: tiles of 128 x 128; 2: tiles of 256 x 256
  int32_t splits;             // runs of the contraction, each a workgroup's; their sums are added afterwards
};

struct GemmParams {
  int32_t M, N, K, G;         // G: groups of the contraction
  int32_t dtype, block;       // of c; rows of b per scale, 1 or 128
  GemmPlan plan;
  const uint8_t *a, *b;
  const float *sa, *sb;
  void* c;
  float* part;                // [splits][M][N]
};
int launch_gemm(const GemmParams& p, void* stream);

}  // namespace gdr
