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
enum GemmKind {
  kGemmFew = 0,     // every row of a, 16 of b
  kGemmSmall = 1,   // tiles of 64 x 128 (rows of a, rows of b)
  kGemmMedium = 2,  // of 128 x 128
  kGemmLarge = 3,   // of 256 x 256
};
constexpr int kFewRows = 32;
struct GemmPlan {
  int32_t kind;
  int32_t splits;   // runs of the contraction, each a workgroup's; their sums are added afterwards
  int32_t copy;     // rows start on 4 bytes: they go to LDS without passing through registers
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
