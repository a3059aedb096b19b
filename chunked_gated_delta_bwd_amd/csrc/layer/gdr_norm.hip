// Root-mean-square norm of rows with the residual's addition, its e4m3 form and
// its backward.
//
// TPR threads hold a row in registers (NV vectors of VEC elements each), so every
// input is read once and every output written once whatever the row needs in
// between: the sum of squares, and for e4m3 the largest magnitude per group.  Narrow
// rows share a wave, and a thread takes UNR rows at a time, so that each has four or
// so 16-byte loads per tensor in flight.  Sums are fp32.  Rows
// need not start on 16 bytes (the device takes vector accesses at the elements' own
// alignment); only a last partial vector goes element by element.
//
// Streaming work, bound by HBM (a large copy on the card measured here moves 4.9
// TB/s): bf16, 8192 x 2048 with residual 28 us (4.8 TB/s), backward 33 us with dw;
// 524288 x 128 50 us (5.4 TB/s), backward 78 us (5.2 TB/s); e4m3 of 32768 x 4096 with
// residual 166 us (5.7 TB/s).  Before narrow rows shared a wave and many threads added
// dw's partial rows, the 524288 x 128 backward took 223 us.  In fp32: 8192 x 2048 with
// residual 50 us (5.4 TB/s), backward 56 us (4.8); 262144 x 128 49 us (5.5), 76 (5.3).
// The backward holds r, dy, dres, w and its share of dw in registers: above 16,384
// channels (1024 threads, 128 registers each) it spills 214 (bf16) or 295 (fp32) of
// them.  8192 x 16384, bf16: 223 us (4.8 TB/s); 8192 x 32768: 1078 us (2.0 TB/s);
// 4096 x 32768, fp32: 886 us (2.4).
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "gdr_layer.h"
#include "gdr_wide.h"

namespace gdr {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126: 1 / scale stays finite

template <typename TIO> constexpr int kVec = 16 / int(sizeof(TIO));

// n of the VEC elements from o on (all of them but at a row's end); the rest is zero
template <typename TIO, int VEC>
__device__ __forceinline__ u32x4 load_raw(const void* b, int64_t o, int n) {
  const TIO* p = static_cast<const TIO*>(b) + o;
  if (n >= VEC) return *reinterpret_cast<const typename Wide<TIO>::T*>(p);
  TIO t[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) t[v] = v < n ? p[v] : TIO(0.f);
  return __builtin_bit_cast(u32x4, t);
}
template <typename TIO, int VEC>
__device__ __forceinline__ void unpack(const u32x4& u, float (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (VEC == 8) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      x[i] = __uint_as_float(u[i]);
    }
  }
}
template <typename TIO, int VEC>
__device__ __forceinline__ void store_n(void* b, int64_t o, int n, const float (&x)[VEC]) {
  TIO* p = static_cast<TIO*>(b) + o;
  if (n >= VEC) {
    u32x4 u;
    if constexpr (VEC == 8) {
      const uint2 lo = pack4_bf16(x[0], x[1], x[2], x[3]), hi = pack4_bf16(x[4], x[5], x[6], x[7]);
      u = u32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(x[i]);
    }
    *reinterpret_cast<typename Wide<TIO>::T*>(p) = u;
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      if (v < n) p[v] = TIO(x[v]);
  }
}
// the weight: fp32, and every vector starts on 16 bytes of it
template <int VEC>
__device__ __forceinline__ void load_w(const float* w, int c, int n, float (&x)[VEC]) {
  if (n >= VEC) {
    if constexpr (VEC == 8) IO<float>::load8(w, c, x);
    else IO<float>::load4(w, c, x);
  } else {
#pragma unroll
    for (int v = 0; v < VEC; ++v) x[v] = v < n ? w[c + v] : 0.f;
  }
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
  const float s = __uint_as_float(bits) / kE4m3Max;
  return s < kMinScale ? kMinScale : s;   // a NaN passes through
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return uint32_t(r);
}

template <typename TIO, int TPR, int NV, int UNR, bool QUANT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm(const NormParams p) {
  constexpr int VEC = kVec<TIO>, BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  constexpr int LANES = TPR < 64 ? TPR : 64;   // of the row's threads in a wave
  static_assert(UNR == 1 || TPR <= 64, "several rows a thread only within a wave");
  __shared__ float red[BS / 64];
  __shared__ uint32_t redm[QUANT ? BS / 64 : 1];
  const int lane = threadIdx.x % TPR, rw = threadIdx.x / TPR;
  const int64_t row0 = int64_t(blockIdx.x) * RPW * UNR + rw;   // then every RPW rows
  u32x4 rx[UNR][NV], rr[UNR][NV];
#pragma unroll
  for (int u = 0; u < UNR; ++u)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + lane) * VEC;
      const int n = row0 + u * RPW < p.rows ? p.width - c : 0;
      const int64_t o = (row0 + u * RPW) * p.width + c;
      rx[u][i] = rr[u][i] = u32x4{0, 0, 0, 0};
      if (n > 0) {
        rx[u][i] = load_raw<TIO, VEC>(p.x, o, n);
        if (p.res) rr[u][i] = load_raw<TIO, VEC>(p.res, o, n);
      }
    }
  float r[UNR][NV][VEC], rstd[UNR];
#pragma unroll
  for (int u = 0; u < UNR; ++u) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float y[VEC];
      unpack<TIO, VEC>(rx[u][i], r[u][i]);
      unpack<TIO, VEC>(rr[u][i], y);
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (p.res) r[u][i][v] += y[v];
        ss += r[u][i][v] * r[u][i][v];
      }
    }
    ss = group_sum<LANES>(ss);
    if constexpr (TPR > 64) {
      if (lane_id() == 0) red[wave_id()] = ss;
      __syncthreads();
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < TPR / 64; ++i) ss += red[i];
    }
    rstd[u] = rsqrtf(ss / float(p.width) + p.eps);
  }
  uint32_t gm[UNR][NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC, n = p.width - c;
    float w[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) w[v] = 1.f;
    if (p.w && n > 0) load_w<VEC>(p.w, c, n, w);
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int64_t o = (row0 + u * RPW) * p.width + c;
      const bool on = n > 0 && row0 + u * RPW < p.rows;
      if (on && p.res_out) store_n<TIO, VEC>(p.res_out, o, n, r[u][i]);
      gm[u][i] = 0;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        r[u][i][v] = r[u][i][v] * rstd[u] * w[v];
        // places past the row's end hold 0 / rms, which may be a NaN of their own
        if (QUANT && v < n) gm[u][i] = max(gm[u][i], __float_as_uint(r[u][i][v]) & 0x7fffffffu);
      }
      if constexpr (!QUANT) {
        if (on) store_n<TIO, VEC>(p.y, o, n, r[u][i]);
      }
    }
  }
  if constexpr (QUANT) {
    // the lanes of one vector index that hold a group of 128 channels (a row with
    // fewer channels than that is one group)
    constexpr int GW = TPR * VEC < 128 ? TPR : 128 / VEC;
    static_assert(TPR * VEC >= 128 || NV == 1, "groups do not cross vector indexes");
    const int groups = p.group ? (p.width + 127) / 128 : 1;
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      const int64_t row = row0 + u * RPW;
      if (p.group == 0) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = max(m, gm[u][i]);
        m = group_max<LANES>(m);
        if constexpr (TPR > 64) {
          if (lane_id() == 0) redm[wave_id()] = m;
          __syncthreads();
#pragma unroll
          for (int i = 0; i < TPR / 64; ++i) m = max(m, redm[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) gm[u][i] = m;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) gm[u][i] = group_max<GW>(gm[u][i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * VEC, n = p.width - c;
        if (n <= 0 || row >= p.rows) continue;
        const float s = scale_of(gm[u][i]);
        if (p.group ? c % 128 == 0 : c == 0) p.scales[row * groups + c / (p.group ? 128 : p.width)] = s;
        // y / s rounded once: the product with the reciprocal and its remainder.  The
        // product alone put one byte in four million on the other side of a border.
        const float inv = 1.f / s, d = s == __builtin_inff() ? 3.0e38f : s;   // y / inf = 0
        float z[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float y = r[u][i][v], p = y * inv;
          // signs as they are so that -0 stays -0; at most 448 (1 + 2^-23), whose byte is 448's
          z[v] = fmaf(-fmaf(p, d, -y), inv, p);
        }
        uint8_t* q = static_cast<uint8_t*>(p.q) + row * p.width + c;
        typedef uint32_t __attribute__((aligned(1))) u32u;
        uint32_t b[VEC / 4];
#pragma unroll
        for (int v = 0; v < VEC / 4; ++v) b[v] = pack_e4m3(z[4 * v], z[4 * v + 1], z[4 * v + 2], z[4 * v + 3]);
        if (n >= VEC) {
          typedef uint32_t __attribute__((ext_vector_type(VEC / 4), aligned(1))) T;
          if constexpr (VEC == 8) *reinterpret_cast<T*>(q) = T{b[0], b[1]};
          else *reinterpret_cast<u32u*>(q) = b[0];
        } else {
#pragma unroll
          for (int v = 0; v < VEC; ++v)
            if (v < n) q[v] = uint8_t(b[v / 4] >> (8 * (v % 4)));
        }
      }
    }
  }
}

// Backward: a workgroup walks the rows in steps of the whole grid and keeps its share
// of dw in registers; the row groups are added in LDS and each workgroup leaves one
// row of partial sums.
template <typename TIO, int TPR, int NV, int UNR>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm_bwd(const NormParams p) {
  constexpr int VEC = kVec<TIO>, BS = TPR > 256 ? TPR : 256, RPW = BS / TPR;
  constexpr int LANES = TPR < 64 ? TPR : 64;
  static_assert(UNR == 1 || TPR <= 64, "several rows a thread only within a wave");
  __shared__ float red[2][2][BS / 64];
  __shared__ float sw[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * VEC : 1];
  const int lane = threadIdx.x % TPR, rw = threadIdx.x / TPR;
  float w[NV][VEC], acc[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + lane) * VEC;
#pragma unroll
    for (int v = 0; v < VEC; ++v) { w[i][v] = 1.f; acc[i][v] = 0.f; }
    if (p.w && c < p.width) load_w<VEC>(p.w, c, p.width - c, w[i]);
  }
  const float inv_width = 1.f / float(p.width);
  int flip = 0;
  for (int64_t first = int64_t(blockIdx.x) * RPW * UNR; first < p.rows; first += int64_t(gridDim.x) * RPW * UNR) {
    const int64_t row0 = first + rw;
    u32x4 rr[UNR][NV], rdy[UNR][NV], rdr[UNR][NV];
#pragma unroll
    for (int u = 0; u < UNR; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * VEC;
        const int n = row0 + u * RPW < p.rows ? p.width - c : 0;
        const int64_t o = (row0 + u * RPW) * p.width + c;
        rr[u][i] = rdy[u][i] = rdr[u][i] = u32x4{0, 0, 0, 0};
        if (n > 0) {
          rr[u][i] = load_raw<TIO, VEC>(p.x, o, n);
          rdy[u][i] = load_raw<TIO, VEC>(p.dy, o, n);
          if (p.dres) rdr[u][i] = load_raw<TIO, VEC>(p.dres, o, n);
        }
      }
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
      float r[NV][VEC], dy[NV][VEC], ss = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<TIO, VEC>(rr[u][i], r[i]);
        unpack<TIO, VEC>(rdy[u][i], dy[i]);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          ss += r[i][v] * r[i][v];
          sd += r[i][v] * dy[i][v] * w[i][v];
        }
      }
      ss = group_sum<LANES>(ss);
      sd = group_sum<LANES>(sd);
      if constexpr (TPR > 64) {
        // the LDS slots alternate, so one barrier a row is enough
        if (lane_id() == 0) { red[flip][0][wave_id()] = ss; red[flip][1][wave_id()] = sd; }
        __syncthreads();
        ss = sd = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) { ss += red[flip][0][i]; sd += red[flip][1][i]; }
        flip ^= 1;
      }
      const float rstd = rsqrtf(ss * inv_width + p.eps);
      const float m = rstd * rstd * (sd * inv_width);
      if (row0 + u * RPW >= p.rows) continue;   // 1 / rms of nothing may be infinite
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * TPR + lane) * VEC, n = p.width - c;
        if (n <= 0) continue;
        float d[VEC], y[VEC];
        unpack<TIO, VEC>(rdr[u][i], y);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          d[v] = rstd * (w[i][v] * dy[i][v] - r[i][v] * m);
          if (p.dres) d[v] += y[v];
          acc[i][v] += dy[i][v] * (r[i][v] * rstd);
        }
        store_n<TIO, VEC>(p.dx, (row0 + u * RPW) * p.width + c, n, d);
      }
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

// dw: the sum of the workgroups' rows, 16 columns a workgroup (so that a narrow
// weight still spreads), 64 runs of rows each added in order
__global__ __launch_bounds__(1024) void k_norm_dw(const float* part, float* dw, int width, int n) {
  __shared__ double s[64][16];
  const int col = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  double d = 0.0;
  if (c < width) {
#pragma unroll 8
    for (int i = g; i < n; i += 64) d += part[int64_t(i) * width + c];
  }
  s[g][col] = d;
  __syncthreads();
  for (int m = 32; m; m >>= 1) {
    if (g < m) s[g][col] += s[g + m][col];
    __syncthreads();
  }
  if (g == 0 && c < width) dw[c] = float(s[0][col]);
}

// Threads per row for a width of n vectors.
struct Plan { int tpr, nv; };
Plan plan_for(int n) {
  if (n <= 2) return {2, 1};
  if (n <= 4) return {4, 1};
  if (n <= 8) return {8, 1};
  if (n <= 16) return {16, 1};
  if (n <= 32) return {32, 1};
  if (n <= 64) return {64, 1};
  if (n <= 128) return {64, 2};
  if (n <= 256) return {64, 4};
  if (n <= 512) return {256, 2};
  if (n <= 1024) return {256, 4};
  if (n <= 2048) return {1024, 2};
  if (n <= 4096) return {1024, 4};
  return {1024, 8};
}
int vectors_of(int width, int dtype) {
  const int v = dtype == GDR_BF16 ? kVec<bf16> : kVec<float>;
  return (width + v - 1) / v;
}
constexpr int unr_for(int tpr, int nv) { return tpr > 64 ? 1 : 4 / nv; }
constexpr int threads_for(int tpr) { return tpr > 256 ? tpr : 256; }
// Rows of a workgroup at a time.
constexpr int rows_for(int tpr, int nv) { return threads_for(tpr) / tpr * unr_for(tpr, nv); }

template <typename TIO, int TPR, int NV>
int launch_fwd(const NormParams& p, hipStream_t s) {
  constexpr int BS = threads_for(TPR), UNR = unr_for(TPR, NV), ROWS = rows_for(TPR, NV);
  const dim3 grid(unsigned((p.rows + ROWS - 1) / ROWS));
  if (p.q) k_norm<TIO, TPR, NV, UNR, true><<<grid, BS, 0, s>>>(p);
  else k_norm<TIO, TPR, NV, UNR, false><<<grid, BS, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

// Workgroups of the backward: as many as stay resident, fewer for few rows.
int partials_for(int64_t rows, int tpr, int nv) {
  const int64_t n = (rows + rows_for(tpr, nv) - 1) / rows_for(tpr, nv);
  return int(n < kNormPartials ? n : kNormPartials);
}

template <typename TIO, int TPR, int NV>
int launch_bwd(const NormParams& p, hipStream_t s) {
  k_norm_bwd<TIO, TPR, NV, unr_for(TPR, NV)><<<dim3(partials_for(p.rows, TPR, NV)), threads_for(TPR), 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename TIO, bool BWD>
int launch_plan(const NormParams& p, hipStream_t s) {
  const Plan pl = plan_for(vectors_of(p.width, p.dtype));
#define GDR_NORM_CASE(T, N) \
  if (pl.tpr == T && pl.nv == N) return BWD ? launch_bwd<TIO, T, N>(p, s) : launch_fwd<TIO, T, N>(p, s);
  GDR_NORM_CASE(2, 1)
  GDR_NORM_CASE(4, 1)
  GDR_NORM_CASE(8, 1)
  GDR_NORM_CASE(16, 1)
  GDR_NORM_CASE(32, 1)
  GDR_NORM_CASE(64, 1)
  GDR_NORM_CASE(64, 2)
  GDR_NORM_CASE(64, 4)
  GDR_NORM_CASE(256, 2)
  GDR_NORM_CASE(256, 4)
  GDR_NORM_CASE(1024, 2)
  GDR_NORM_CASE(1024, 4)
  if constexpr (sizeof(TIO) == 4) { GDR_NORM_CASE(1024, 8) }
#undef GDR_NORM_CASE
  return static_cast<int>(hipErrorInvalidConfiguration);
}

template <bool BWD>
int launch_any(const NormParams& p, hipStream_t s) {
  return p.dtype == GDR_BF16 ? launch_plan<bf16, BWD>(p, s) : launch_plan<float, BWD>(p, s);
}

}  // namespace

int64_t norm_fwd_blocks(int64_t rows, int32_t width, int32_t dtype) {
  const Plan pl = plan_for(vectors_of(width, dtype));
  return (rows + rows_for(pl.tpr, pl.nv) - 1) / rows_for(pl.tpr, pl.nv);
}

int norm_fwd_threads(int32_t width, int32_t dtype) { return threads_for(plan_for(vectors_of(width, dtype)).tpr); }

int norm_bwd_partials(int64_t rows, int32_t width, int32_t dtype) {
  const Plan pl = plan_for(vectors_of(width, dtype));
  return partials_for(rows, pl.tpr, pl.nv);
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
  k_norm_dw<<<dim3((p.width + 15) / 16), 1024, 0, s>>>(p.part, p.dw, p.width,
                                                       norm_bwd_partials(p.rows, p.width, p.dtype));
  return static_cast<int>(hipGetLastError());
}

}  // namespace gdr
