// Host side of the e4m3 product and of the quantisation that makes its operands (see
// gdr.h): argument checks, the choice of the tiles and the launch sequences.  Nothing
// here allocates or synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "gdr_check.h"
#include "gdr_gemm.h"
#include "gdr_layer.h"

namespace {

using namespace gdr::check;
using gdr::set_error;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

gdr_status check_quant_shape(const gdr_quant_shape* s) {
  if (!s) return set_error(GDR_EINVAL, "shape is NULL");
  if (s->dtype != GDR_BF16 && s->dtype != GDR_F32) return set_error(GDR_EINVAL, "unknown dtype %d", s->dtype);
  if (s->rows < 0 || s->cols < 0) return set_error(GDR_EINVAL, "bad rows/cols");
  if (s->block != 1 && s->block != gdr::kGroup) return set_error(GDR_EUNSUPPORTED, "block %d not in {1, 128}", s->block);
  if (s->transpose != 0 && s->transpose != 1) return set_error(GDR_EINVAL, "transpose %d must be 0 or 1", s->transpose);
  constexpr int64_t most = int64_t(1) << 31;
  if (s->rows >= most || s->cols >= most ||
      ceil_div(s->rows, gdr::kGroup) * ceil_div(s->cols, gdr::kGroup) * 256 >= gdr::kMaxThreads)
    return set_error(GDR_EUNSUPPORTED, "matrix too large for one launch");
  return GDR_OK;
}

gdr_status check_gemm_shape(const gdr_gemm_shape* s) {
  if (!s) return set_error(GDR_EINVAL, "shape is NULL");
  if (s->dtype != GDR_BF16 && s->dtype != GDR_F32) return set_error(GDR_EINVAL, "unknown dtype %d", s->dtype);
  if (s->M < 0 || s->N < 0 || s->K < 1) return set_error(GDR_EINVAL, "bad M/N/K");
  if (s->block != 1 && s->block != gdr::kGroup) return set_error(GDR_EUNSUPPORTED, "block %d not in {1, 128}", s->block);
  if (s->M > (1 << 30) || s->N > (1 << 30) || s->K > (1 << 30) ||
      ceil_div(s->M, 128) * ceil_div(s->N, 128) >= (int64_t(1) << 19))
    return set_error(GDR_EUNSUPPORTED, "product too large for one launch");
  return GDR_OK;
}

// The cut, by what was measured in us (M x N x K; bf16 results unless f32 is said):
//                              64 x 128   128 x 128   256 x 256
//   512 x 4096 x 4096             22.3        32.1         -
//   1024 x 4096 x 4096            30.5        34.4         -
//   2048 x 2048 x 2048            17.4        19.0        28.9
//   2048 x 2048 x 2048, f32       25.9        31.6         -
//   2304 x 2048 x 2048            26.3        21.8         -
//   2560 x 2048 x 2048, f32       38.5        40.4         -
//   3500 x 2048 x 2048, f32       45.5        42.6         -
//   4096 x 2048 x 8192            98.5        72.5         -
//   4096 x 2048 x 8192, rows     118          94.2       143
//   2048 x 4096 x 4096            55.5        40.5        52.1
//   2560 x 4096 x 4096             -          68.4        56.3
//   3584 x 4096 x 4096             -          83.8        69.0
//   4096 x 4096 x 4096            97.3        79.5        68.3
//   4400 x 4096 x 4096             -         108.2       108.7
//   10000 x 4096 x 4096            -         199         169
//   4096 x 4096 x 512             24.1        19.0        18.1
//   8192 x 4096 x 256             35.3        26.0        31.9
//   32768 x 4096 x 4096          843         655         519
// Two workgroups of 64 x 128 fit a compute unit: up to 512 they run together, and are the
// shorter ones.  With fp32 results, where the instructions take twice as long, so they are a
// little beyond.
// One of 256 x 256 fills a compute unit as two of 128 x 128 do; a round of them takes about
// 4 / 3 of the other's time.
// A split contraction pays where few workgroups leave most compute units idle: 64 x 4096 x
// 4096 with 32 workgroups 12.9 in 4 runs, 14.1 in 2, 16.2 as one for every 16 rows of b;
// 256 x 4096 x 4096 with 128 workgroups 17.3 whole, 21.4 in 2 runs.  Rows that pass through
// registers take a split further: 1000 x 2050 x 4102, f32, 53.8 whole, 51.3 in 2 runs, and
// 500 x 1030 x 2046 25.8 and 20.6, where the K of 4096 takes 37.9 whole, 42.7 in 2.  Rows on
// 4 bytes copied to LDS: 1000 x 2050 x 4100, f32, 46.8, through registers 48.2.
gdr::GemmPlan gemm_plan(const gdr_gemm_shape* s) {
  const int64_t groups = ceil_div(s->K, gdr::kGroup);
  if (s->M <= gdr::kFewRows) return {gdr::kGemmFew, 1, 0};
  const int32_t copy = s->K % 4 == 0 && s->K <= (1 << 22);   // 256 rows within 32 bits
  const int64_t large = ceil_div(ceil_div(s->M, 256) * ceil_div(s->N, 256), 256);
  const int64_t medium = ceil_div(ceil_div(s->M, 128) * ceil_div(s->N, 128), 512);
  if (copy && s->dtype == GDR_BF16 && groups >= 4 && 4 * large < 3 * medium) return {gdr::kGemmLarge, 1, copy};
  const int64_t tiles = ceil_div(s->M, 64) * ceil_div(s->N, 128);
  if (tiles > (s->dtype == GDR_BF16 ? 512 : 768)) return {gdr::kGemmMedium, 1, copy};
  const int64_t splits = std::min<int64_t>(tiles <= 64 ? 4 : !copy && tiles <= 512 ? 2 : 1, groups / 8);
  if (splits < 2) return {gdr::kGemmSmall, 1, copy};
  // no run without a group: the last one may be shorter than the others
  return {gdr::kGemmSmall, int32_t(ceil_div(groups, ceil_div(groups, splits))), copy};
}

size_t gemm_ws(const gdr_gemm_shape* s) {
  const gdr::GemmPlan plan = gemm_plan(s);
  return plan.splits > 1 ? align256(size_t(plan.splits) * size_t(s->M) * size_t(s->N) * 4) : 0;
}

}  // namespace

extern "C" {

gdr_status gdr_quant(const gdr_quant_shape* shape, const void* x, void* q, float* scales, void* stream) {
  gdr_status st = check_quant_shape(shape);
  if (st != GDR_OK) return st;
  const bool any = shape->rows > 0 && shape->cols > 0;
  const Arg a[] = {{x, "x", any}, {q, "q", any}, {scales, "scales", any}};
  if ((st = check_ptrs(a, 3)) != GDR_OK) return st;
  gdr::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = shape->rows; p.cols = shape->cols;
  p.dtype = shape->dtype; p.block = shape->block; p.transpose = shape->transpose;
  p.x = x; p.q = q; p.scales = scales;
  return hip_status(gdr::launch_quant(p, stream), "quantisation kernel");
}

gdr_status gdr_gemm_workspace_bytes(const gdr_gemm_shape* shape, size_t* bytes) {
  const gdr_status st = check_gemm_shape(shape);
  if (st != GDR_OK) return st;
  if (!bytes) return set_error(GDR_EINVAL, "bytes is NULL");
  *bytes = gemm_ws(shape);
  return GDR_OK;
}

gdr_status gdr_gemm(const gdr_gemm_shape* shape, const void* a, const float* a_scales, const void* b,
                    const float* b_scales, void* ws, size_t ws_bytes, void* c, void* stream) {
  gdr_status st = check_gemm_shape(shape);
  if (st != GDR_OK) return st;
  const bool any = shape->M > 0 && shape->N > 0;
  const Arg args[] = {{a, "a", any}, {a_scales, "a_scales", any}, {b, "b", any}, {b_scales, "b_scales", any}, {c, "c", any}};
  if ((st = check_ptrs(args, 5)) != GDR_OK) return st;
  if ((st = check_ws(gemm_ws(shape), ws, ws_bytes)) != GDR_OK) return st;
  gdr::GemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = shape->M; p.N = shape->N; p.K = shape->K; p.G = int32_t(ceil_div(shape->K, gdr::kGroup));
  p.dtype = shape->dtype; p.block = shape->block; p.plan = gemm_plan(shape);
  p.a = static_cast<const uint8_t*>(a); p.b = static_cast<const uint8_t*>(b);
  p.sa = a_scales; p.sb = b_scales; p.c = c; p.part = static_cast<float*>(ws);
  return hip_status(gdr::launch_gemm(p, stream), "product kernel");
}

}  // extern "C"
