// A matrix, or its transpose, as e4m3 with a scale for each 128 elements of a row of the
// result, or for each block of 128 x 128 (gdr_quant).
//
// A workgroup holds a tile of 128 x 128 elements in registers (thread (rg, cg) the rows
// 8 rg .. + 7 and columns 8 cg .. + 7), so that x is read once whatever direction the
// scales run in: largest magnitudes of rows are reduced over 16 lanes, of columns over 4
// lanes and 4 waves, of the block over both.  A transposed tile turns around in LDS as
// bytes.  Streaming work, bound by HBM: 4096 x 4096 bf16 to blocks, transposed, 11.2 us
// (50 MB, 4.5 TB/s); 8192 x 4096, rows, 27.3 (the kernel; 101 MB, 3.7 TB/s) and transposed
// 23.3 (4.4 TB/s).
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "gdr_gemm.h"
#include "gdr_wide.h"

namespace gdr {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: 1 / scale stays finite

typedef uint32_t __attribute__((ext_vector_type(2), aligned(1))) u32x2u;
typedef uint32_t __attribute__((ext_vector_type(4), aligned(1))) u32x4u;

// n of the 8 elements at p (all of them but at a row's end); the rest is zero
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float (&x)[8]) {
  if (n >= 8) {
    if constexpr (sizeof(T) == 2) {
      const u32x4 u = *reinterpret_cast<const typename Wide<T>::T*>(p);
      IO<bf16>::unpack8(u, x);
    } else {
      const u32x4 a = *reinterpret_cast<const typename Wide<T>::T*>(p), b = *reinterpret_cast<const typename Wide<T>::T*>(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(a[i]);
        x[4 + i] = __uint_as_float(b[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? float(p[i]) : 0.f;
  }
}

// Magnitudes as the bits of |x|: integer order is their order, with NaN above every number.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t xor_max(uint32_t x, int m) { return max(x, uint32_t(__shfl_xor(int(x), m, 64))); }

__device__ __forceinline__ float scale_of(uint32_t bits) {
  const float s = __uint_as_float(bits) / kE4m3Max;
  return s < kMinScale ? kMinScale : s;   // a NaN passes through
}
// x / s rounded once: the product with the reciprocal and its remainder; x / inf = 0
__device__ __forceinline__ float quotient(float x, float inv, float s) {
  const float p = x * inv;
  return fmaf(-fmaf(p, s == __builtin_inff() ? 3.0e38f : s, -x), inv, p);
}
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return uint32_t(r);
}

// ROWS: scales for 128 elements of a row of the result (a column of x, transposed); else
// for the block.
template <typename T, bool TRANS, bool ROWS>
__global__ __launch_bounds__(256) void k_quant(const QuantParams p) {
  constexpr bool COLMAX = TRANS && ROWS;
  __shared__ uint32_t red[COLMAX ? 4 : 1][128];
  __shared__ __attribute__((aligned(16))) uint2 turn[TRANS ? 128 * 16 : 1];
  const int lane = lane_id(), wave = wave_id(), cg = lane & 15, rg = 4 * wave + (lane >> 4);
  const int64_t tiles_c = (p.cols + 127) / 128;
  const int64_t tr = blockIdx.x / tiles_c, tc = blockIdx.x % tiles_c;
  const int64_t row0 = tr * 128 + 8 * rg, col0 = tc * 128 + 8 * cg;
  const int nr = int(min(int64_t(8), p.rows - row0)), nc = int(min(int64_t(8), p.cols - col0));   // <= 0: outside
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<T>(static_cast<const T*>(p.x) + (row0 + i) * p.cols + col0, i < nr ? nc : 0, x[i]);
  if constexpr (!COLMAX) {
    uint32_t m[8], all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m[i] = max(m[i], mag(x[i][j]));
      if constexpr (ROWS) {
#pragma unroll
        for (int s = 1; s < 16; s <<= 1) m[i] = xor_max(m[i], s);
      }
      all = max(all, m[i]);
    }
    if constexpr (!ROWS) {
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) all = xor_max(all, s);
      if (lane == 0) red[0][wave] = all;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 4; ++w) all = max(all, red[0][w]);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = all;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = scale_of(m[i]), inv = 1.f / s;
      if (ROWS && cg == 0 && i < nr) p.scales[(row0 + i) * tiles_c + tc] = s;
      if (!ROWS && i == 0 && threadIdx.x == 0)
        p.scales[TRANS ? tc * ((p.rows + 127) / 128) + tr : tr * tiles_c + tc] = s;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = quotient(x[i][j], inv, s);
    }
  } else {
    uint32_t m[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = max(m[j], mag(x[i][j]));
      m[j] = xor_max(xor_max(m[j], 16), 32);
      if (lane < 16) red[wave][8 * cg + j] = m[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int w = 0; w < 4; ++w) m[j] = max(m[j], red[w][8 * cg + j]);
      const float s = scale_of(m[j]), inv = 1.f / s;
      if (rg == 0 && j < nc) p.scales[(col0 + j) * ((p.rows + 127) / 128) + tr] = s;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i][j] = quotient(x[i][j], inv, s);
    }
  }
  uint8_t* q = static_cast<uint8_t*>(p.q);
  if constexpr (!TRANS) {
    if (nc <= 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= nr) break;
      const uint32_t lo = pack_e4m3(x[i][0], x[i][1], x[i][2], x[i][3]), hi = pack_e4m3(x[i][4], x[i][5], x[i][6], x[i][7]);
      uint8_t* d = q + (row0 + i) * p.cols + col0;
      if (nc == 8) {
        *reinterpret_cast<u32x2u*>(d) = u32x2u{lo, hi};
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < nc) d[j] = uint8_t((j < 4 ? lo : hi) >> (8 * (j % 4)));
      }
    }
  } else {
    // 8 bytes (rows 8 rg .. + 7) of column 8 cg + j at place rg ^ cg of its 16: the writes
    // of a wave, and the 16-byte reads below, meet different banks
#pragma unroll
    for (int j = 0; j < 8; ++j)
      turn[(8 * cg + j) * 16 + (rg ^ cg)] = uint2{pack_e4m3(x[0][j], x[1][j], x[2][j], x[3][j]),
                                                  pack_e4m3(x[4][j], x[5][j], x[6][j], x[7][j])};
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = i * 256 + threadIdx.x, c = id >> 3, piece = id & 7;   // 16 rows of column c
      const int64_t col = tc * 128 + c, r = tr * 128 + 16 * piece;
      if (col >= p.cols || r >= p.rows) continue;
      const int s = (c >> 3) & 15;
      const uint4 two = *reinterpret_cast<const uint4*>(&turn[c * 16 + ((2 * piece) ^ (s & 14))]);
      const u32x4 v = s & 1 ? u32x4{two.z, two.w, two.x, two.y} : u32x4{two.x, two.y, two.z, two.w};
      uint8_t* d = q + col * p.rows + r;
      const int n = int(min(int64_t(16), p.rows - r));
      if (n == 16) {
        *reinterpret_cast<u32x4u*>(d) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < n) d[j] = uint8_t(v[j / 4] >> (8 * (j % 4)));
      }
    }
  }
}

template <typename T>
int launch_type(const QuantParams& p, hipStream_t s) {
  const unsigned grid = unsigned(((p.rows + 127) / 128) * ((p.cols + 127) / 128));
  const bool rows = p.block == 1;
  if (p.transpose) {
    if (rows) k_quant<T, true, true><<<grid, 256, 0, s>>>(p);
    else k_quant<T, true, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (rows) k_quant<T, false, true><<<grid, 256, 0, s>>>(p);
    else k_quant<T, false, false><<<grid, 256, 0, s>>>(p);
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_quant(const QuantParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.rows == 0 || p.cols == 0) return 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == GDR_BF16 ? launch_type<bf16>(p, s) : launch_type<float>(p, s);
}

}  // namespace gdr
