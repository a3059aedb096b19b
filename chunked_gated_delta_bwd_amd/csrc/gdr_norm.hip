// Root-mean-square norm of rows with the residual's addition, its e4m3 form and
// its backward.
//
// TPR threads hold a row in registers (NV vectors of VEC elements each), so every
// input is read once and every output written once whatever the row needs in
// between: the sum of squares, and for e4m3 the largest magnitude per group.
// Sums are fp32.  Streaming work, bound by HBM.
#include <hip/hip_runtime.h>

#include "gdr_device.h"
#include "gdr_layer.h"

namespace gdr {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: 1 / scale stays finite

template <typename TIO, int VEC>
__device__ __forceinline__ void load_v(const void* b, int64_t o, float (&x)[VEC]) {
  if constexpr (VEC == 8) IO<TIO>::load8(b, o, x);
  else if constexpr (VEC == 4) IO<TIO>::load4(b, o, x);
  else x[0] = IO<TIO>::load1(b, o);
}
template <typename TIO, int VEC>
__device__ __forceinline__ void store_v(void* b, int64_t o, const float (&x)[VEC]) {
  if constexpr (VEC == 8) IO<TIO>::store8(b, o, x);
  else if constexpr (VEC == 4) IO<TIO>::store4(b, o, x[0], x[1], x[2], x[3]);
  else IO<TIO>::store1(b, o, x[0]);
}

// Sum over the TPR threads of a row, on each of them.  `red`: one float per wave
// and call slot.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = group_sum<(TPR < 64 ? TPR : 64)>(x);
  if constexpr (TPR > 64) {
    if (lane_id() == 0) red[wave_id()] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) x += red[i];
  }
  return x;
}

// Largest magnitude as the bits of |x|: integer order is the order of the
// magnitudes, with NaN above every number.
template <int W>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
#pragma unroll
  for (int m = W / 2; m >= 1; m >>= 1) x = max(x, uint32_t(__shfl_xor(int(x), m, 64)));
  return x;
}

__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float m = __uint_as_float(bits);
  const float s = m / kE4m3Max;
  return s < kMinScale ? kMinScale : s;   // a NaN passes through
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return uint32_t(r);
}

template <typename TIO, int VEC, int TPR, int NV, bool QUANT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm(const NormParams p) {
  constexpr int BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  __shared__ float red[BS / 64];
  __shared__ uint32_t redm[QUANT ? BS / 64 : 1];
  __shared__ uint32_t gmax[QUANT && VEC == 1 ? RPW : 1][QUANT && VEC == 1 ? (TPR * NV + 127) / 128 : 1];
  const int lane = threadIdx.x % TPR, rw = threadIdx.x / TPR;
  const int64_t row = int64_t(blockIdx.x) * RPW + rw;
  const bool on = row < p.rows;
  const int64_t base = row * p.width;
  float r[NV][VEC], ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
    if (on && c < p.width) {
      load_v<TIO, VEC>(p.x, base + c, r[i]);
      if (p.res) {
        float y[VEC];
        load_v<TIO, VEC>(p.res, base + c, y);
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[i][v] += y[v];
      }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) r[i][v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) ss += r[i][v] * r[i][v];
  }
  ss = row_sum<TPR>(ss, red);
  const float rstd = rsqrtf(ss / float(p.width) + p.eps);
  uint32_t amax = 0, gm[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
    const bool in = on && c < p.width;
    float w[VEC];
    if (in) {
      if (p.res_out) store_v<TIO, VEC>(p.res_out, base + c, r[i]);
      if (p.w) load_v<float, VEC>(p.w, c, w);
      else
#pragma unroll
        for (int v = 0; v < VEC; ++v) w[v] = 1.f;
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) w[v] = 0.f;
    }
    gm[i] = 0;
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      r[i][v] = in ? r[i][v] * rstd * w[v] : 0.f;
      if constexpr (QUANT) gm[i] = max(gm[i], __float_as_uint(r[i][v]) & 0x7fffffffu);
    }
    amax = max(amax, gm[i]);
    if constexpr (!QUANT) {
      if (in) store_v<TIO, VEC>(p.y, base + c, r[i]);
    }
  }
  if constexpr (QUANT) {
    // gm[i] becomes the group's maximum
    if (p.group == 0) {
      amax = group_max<(TPR < 64 ? TPR : 64)>(amax);
      if constexpr (TPR > 64) {
        if (lane_id() == 0) redm[wave_id()] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) amax = max(amax, redm[i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) gm[i] = amax;
      if (on && lane == 0) p.scales[row] = scale_of(amax);
    } else if constexpr (VEC > 1) {
      // a group of 128 channels is 128 / VEC neighbouring lanes
      static_assert(TPR * VEC >= 128, "a group spans lanes of one vector index");
      const int groups = (p.width + 127) / 128;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        gm[i] = group_max<128 / VEC>(gm[i]);
        const int c = (i * TPR + lane) * VEC;
        if (on && c < p.width && c % 128 == 0) p.scales[row * groups + c / 128] = scale_of(gm[i]);
      }
    } else {
      const int groups = (p.width + 127) / 128;
      for (int i = lane; i < groups; i += TPR) gmax[rw][i] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * TPR + lane;
        if (c < p.width) atomicMax(&gmax[rw][c / 128], gm[i]);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * TPR + lane;
        if (c < p.width) gm[i] = gmax[rw][c / 128];
        if (on && c < p.width && c % 128 == 0) p.scales[row * groups + c / 128] = scale_of(gm[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      if (!(on && c < p.width)) continue;
      const float s = scale_of(gm[i]);
      float z[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float t = r[i][v] / s;
        z[v] = t != t ? t : fminf(fmaxf(t, -kE4m3Max), kE4m3Max);
      }
      uint8_t* q = static_cast<uint8_t*>(p.q) + base + c;
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(q) = make_uint2(pack_e4m3(z[0], z[1], z[2], z[3]), pack_e4m3(z[4], z[5], z[6], z[7]));
      else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(q) = pack_e4m3(z[0], z[1], z[2], z[3]);
      else q[0] = uint8_t(pack_e4m3(z[0], 0.f, 0.f, 0.f));
    }
  }
}

// Backward: a workgroup walks rows blockIdx.x, + gridDim.x, ... (in units of its
// RPW rows) and keeps its share of dw in registers; the row groups are added in
// LDS and each workgroup leaves one row of partial sums.
template <typename TIO, int VEC, int TPR, int NV>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm_bwd(const NormParams p) {
  constexpr int BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  __shared__ float red[2][2][BS / 64];
  __shared__ float sw[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * VEC : 1];
  const int lane = threadIdx.x % TPR, rw = threadIdx.x / TPR;
  float w[NV][VEC], acc[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) { w[i][v] = 1.f; acc[i][v] = 0.f; }
    if (c < p.width && p.w) load_v<float, VEC>(p.w, c, w[i]);
  }
  int flip = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * RPW; row0 < p.rows; row0 += int64_t(gridDim.x) * RPW, flip ^= 1) {
    const int64_t row = row0 + rw;
    const bool on = row < p.rows;
    const int64_t base = row * p.width;
    float r[NV][VEC], dy[NV][VEC], ss = 0.f, sd = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      if (on && c < p.width) {
        load_v<TIO, VEC>(p.x, base + c, r[i]);
        load_v<TIO, VEC>(p.dy, base + c, dy[i]);
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) r[i][v] = dy[i][v] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        ss += r[i][v] * r[i][v];
        sd += r[i][v] * dy[i][v] * w[i][v];
      }
    }
    // two sums a row; the LDS slots alternate, so one barrier per row is enough
    ss = group_sum<(TPR < 64 ? TPR : 64)>(ss);
    sd = group_sum<(TPR < 64 ? TPR : 64)>(sd);
    if constexpr (TPR > 64) {
      if (lane_id() == 0) { red[flip][0][wave_id()] = ss; red[flip][1][wave_id()] = sd; }
      __syncthreads();
      ss = sd = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 64; ++i) { ss += red[flip][0][i]; sd += red[flip][1][i]; }
    }
    const float rstd = rsqrtf(ss / float(p.width) + p.eps);
    const float m = rstd * rstd * (sd / float(p.width));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      if (!(on && c < p.width)) continue;
      float d[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        d[v] = rstd * (w[i][v] * dy[i][v] - r[i][v] * m);
        acc[i][v] += dy[i][v] * (r[i][v] * rstd);
      }
      if (p.dres) {
        float y[VEC];
        load_v<TIO, VEC>(p.dres, base + c, y);
#pragma unroll
        for (int v = 0; v < VEC; ++v) d[v] += y[v];
      }
      store_v<TIO, VEC>(p.dx, base + c, d);
    }
  }
  if (!p.part) return;
  float* part = p.part + int64_t(blockIdx.x) * p.width;
  if constexpr (RPW == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const int c = (i * TPR + lane) * VEC + v;
        if (c < p.width) part[c] = acc[i][v];
      }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int v = 0; v < VEC; ++v) sw[rw][(i * TPR + lane) * VEC + v] = acc[i][v];
    __syncthreads();
    for (int c = threadIdx.x; c < p.width; c += BS) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < RPW; ++i) d += sw[i][c];
      part[c] = d;
    }
  }
}

// dw: the sum of the workgroups' rows, 64 columns a workgroup, four runs of rows
// each added in order
__global__ __launch_bounds__(256) void k_norm_dw(const float* part, float* dw, int width, int n) {
  __shared__ double s[4][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), g = threadIdx.x >> 6;
  double d = 0.0;
  if (c < width)
    for (int i = g; i < n; i += 4) d += part[int64_t(i) * width + c];
  s[g][threadIdx.x & 63] = d;
  __syncthreads();
  if (g == 0 && c < width) dw[c] = float(s[0][threadIdx.x] + s[1][threadIdx.x] + s[2][threadIdx.x] + s[3][threadIdx.x]);
}

// Threads per row and vectors per thread for a width: whole waves once a row
// fills one, four vectors a thread before more threads.
struct Plan { int tpr, nv; };
Plan plan_for(int width, int vec) {
  const int n = (width + vec - 1) / vec;
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  if (n <= 256) return {64, 4};
  if (n <= 1024) return {256, 4};
  if (n <= 4096) return {1024, 4};
  return {1024, vec == 1 ? 32 : 8};
}

int vec_of(int width, int dtype) {
  const int v = dtype == GDR_BF16 ? 8 : 4;
  return width % v == 0 ? v : 1;
}

template <typename TIO, int VEC, int TPR, int NV>
int launch_fwd(const NormParams& p, hipStream_t s) {
  constexpr int BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  const dim3 grid(unsigned((p.rows + RPW - 1) / RPW));
  if (p.q) k_norm<TIO, VEC, TPR, NV, true><<<grid, BS, 0, s>>>(p);
  else k_norm<TIO, VEC, TPR, NV, false><<<grid, BS, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

int partials_for(int64_t rows, int rpw) {
  const int64_t n = (rows + rpw - 1) / rpw;
  return int(n < kNormPartials ? n : kNormPartials);
}

template <typename TIO, int VEC, int TPR, int NV>
int launch_bwd(const NormParams& p, hipStream_t s) {
  constexpr int BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  k_norm_bwd<TIO, VEC, TPR, NV><<<dim3(partials_for(p.rows, RPW)), BS, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename TIO, int VEC, bool BWD>
int launch_plan(const NormParams& p, hipStream_t s) {
  const Plan pl = plan_for(p.width, VEC);
#define GDR_NORM_CASE(T, N) \
  if (pl.tpr == T && pl.nv == N) return BWD ? launch_bwd<TIO, VEC, T, N>(p, s) : launch_fwd<TIO, VEC, T, N>(p, s);
  GDR_NORM_CASE(32, 1)
  GDR_NORM_CASE(64, 1)
  GDR_NORM_CASE(64, 2)
  GDR_NORM_CASE(64, 4)
  GDR_NORM_CASE(256, 4)
  GDR_NORM_CASE(1024, 4)
  if constexpr (VEC == 1) { GDR_NORM_CASE(1024, 32) }
  else if constexpr (VEC == 4) { GDR_NORM_CASE(1024, 8) }
#undef GDR_NORM_CASE
  return static_cast<int>(hipErrorInvalidConfiguration);
}

template <bool BWD>
int launch_any(const NormParams& p, hipStream_t s) {
  if (p.dtype == GDR_BF16)
    return p.width % 8 == 0 ? launch_plan<bf16, 8, BWD>(p, s) : launch_plan<bf16, 1, BWD>(p, s);
  return p.width % 4 == 0 ? launch_plan<float, 4, BWD>(p, s) : launch_plan<float, 1, BWD>(p, s);
}

}  // namespace

int norm_bwd_partials(int64_t rows, int32_t width, int32_t dtype) {
  const Plan pl = plan_for(width, vec_of(width, dtype));
  return partials_for(rows, pl.tpr > 256 ? 1 : 256 / pl.tpr);
}

int launch_norm(const NormParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.rows == 0) return 0;
  return launch_any<false>(p, reinterpret_cast<hipStream_t>(stream));
}

int launch_norm_bwd(const NormParams& p, void* stream) {
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  int e = p.rows ? launch_any<true>(p, s) : 0;
  if (e || !p.dw) return e;
  k_norm_dw<<<dim3((p.width + 63) / 64), 256, 0, s>>>(p.part, p.dw, p.width,
                                                       norm_bwd_partials(p.rows, p.width, p.dtype));
  return static_cast<int>(hipGetLastError());
}

}  // namespace gdr
