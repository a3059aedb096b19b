// Product of e4m3 matrices with a scale for each 128 of the contraction (gdr_gemm).
//
//   c[m][n] = sum_g sa[m][g] sb[n][g] sum_{k in g} a[m][k] b[n][k]
// The inner sum over a group's 128 elements is matrix instructions alone (32x32x64, two
// a group), started from zero; what they leave is scaled and added in fp32, so that the
// scales may be any numbers.  b's rows are the instruction's rows and a's its columns:
// a lane then holds sums of one row of a, whose scale is one register, and b's scale is
// the same for all of them where it belongs to a block of 128 rows.
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "../gdr_lds.h"
#include "gdr_gemm.h"
#include "gdr_wide.h"

namespace gdr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t __attribute__((ext_vector_type(4), aligned(1))) u32x4u;

// Sum over 64 of the contraction (32x32) or 128 (16x16): a lane's 32 bytes of its row.
// EXACT: the e4m3 instructions align the products that they add together to the largest
// of them and drop what lies 2^-13 below it (found by adding 2^-s to 1: from s = 14 on a
// neighbour's 2^-s is gone, whichever e4m3 instruction is used).  On quantised normal
// data that leaves a sum with an error of 1.3e-5 of its size, far below the rounding of a
// bf16 result (1.7e-3) but not of an fp32 one: there the bytes become bf16, which holds
// them and whose instructions add in fp32 (9e-9), at half the rate.
__device__ __forceinline__ bf16x8 to_bf16x8(int lo, int hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return __builtin_bit_cast(bf16x8, u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                                          __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)});
}
template <bool EXACT> struct Bytes { typedef i32x8 T; };
template <> struct Bytes<true> { struct T { bf16x8 v[4]; }; };

template <bool EXACT>
__device__ __forceinline__ typename Bytes<EXACT>::T operand(i32x8 u) {
  if constexpr (EXACT) {
    typename Bytes<true>::T t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t.v[i] = to_bf16x8(u[2 * i], u[2 * i + 1]);
    return t;
  } else {
    return u;
  }
}
__device__ __forceinline__ f32x16 mul32(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mul16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mul32(const Bytes<true>::T& a, const Bytes<true>::T& b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}
__device__ __forceinline__ f32x4 mul16(const Bytes<true>::T& a, const Bytes<true>::T& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mma(a.v[i], b.v[i], c);
  return c;
}

// n of the 16 bytes at p, the rest zero
__device__ __forceinline__ u32x4 bytes16(const uint8_t* p, int n) {
  if (n >= 16) return *reinterpret_cast<const u32x4u*>(p);
  u32x4 v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) v[i / 4] |= uint32_t(p[i]) << (8 * (i % 4));
  return v;
}

// n of the VEC results for c[at ..]
template <typename T, int VEC>
__device__ __forceinline__ void put(void* c, int64_t at, int n, const float (&x)[VEC]) {
  T* d = static_cast<T*>(c) + at;
  if (n >= VEC) {
#pragma unroll
    for (int i = 0; i < VEC; i += 16 / int(sizeof(T))) {
      if constexpr (sizeof(T) == 2) {
        const uint2 lo = pack4_bf16(x[i], x[i + 1], x[i + 2], x[i + 3]), hi = pack4_bf16(x[i + 4], x[i + 5], x[i + 6], x[i + 7]);
        *reinterpret_cast<typename Wide<T>::T*>(d + i) = u32x4{lo.x, lo.y, hi.x, hi.y};
      } else {
        *reinterpret_cast<typename Wide<T>::T*>(d + i) = u32x4{__float_as_uint(x[i]), __float_as_uint(x[i + 1]),
                                                               __float_as_uint(x[i + 2]), __float_as_uint(x[i + 3])};
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) d[i] = T(x[i]);
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// LDS rows of 128 bytes; piece p (16 bytes) of row r at piece p ^ (r / 2 mod 8): the 16
// lanes that a 16-byte read serves together lie in rows of which no two of one parity
// (one half of the banks) share r / 2 mod 8
__device__ __forceinline__ int place(int r, int p) { return r * 128 + ((p ^ ((r >> 1) & 7)) << 4); }
__device__ __forceinline__ i32x8 frag(const char* t, int r, int kk) {
  const int p = 4 * kk + 2 * (lane_id() >> 5);
  const u32x4 lo = *reinterpret_cast<const u32x4*>(t + place(r, p));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(t + place(r, p + 1));
  return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Workgroup ids go round-robin over the 8 XCDs: each takes a run of tiles, and a run goes
// through stripes of 8 row tiles, so that an XCD's L2 holds what its workgroups share.
__device__ __forceinline__ void tile_at(int id, int tm, int tn, int& m, int& n) {
  const int total = tm * tn, each = total / 8, more = total % 8, x = id % 8;
  const int t = x * each + min(x, more) + id / 8;
  const int stripe = 8 * tn, s = t / stripe, rows = min(8, tm - 8 * s), r = t - s * stripe;
  m = 8 * s + r % rows;
  n = r / rows;
}

template <bool SHORT> struct Off { typedef uint32_t T; };
template <> struct Off<false> { typedef int64_t T; };

// T: what the sums are stored as (fp32 for the partial sums of a split contraction).
// ROWS: b has a scale for each row.  DMA: rows start on 16 bytes.
template <typename T, int BM, int BN, int WM, int WN, bool EXACT, bool ROWS, bool DMA>
__global__ __launch_bounds__(64 * WM * WN) void k_gemm(const GemmParams p) {
  constexpr int NT = 64 * WM * WN, MT = BM / WM / 32, QT = BN / WN / 32;
  constexpr int LA = BM / 8 / (WM * WN), LB = BN / 8 / (WM * WN);   // 1 KB loads a wave
  static_assert(BM + BN <= NT || BM + BN == 2 * NT, "scales per thread");
  constexpr int SC = (BM + BN + NT - 1) / NT;
  __shared__ __attribute__((aligned(1024))) char as[2][BM * 128], bs[2][BN * 128];
  __shared__ float ss[2][BM + BN];
  int tm, tn;
  tile_at(int(blockIdx.x), (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int per = (p.G + p.plan.splits - 1) / p.plan.splits, g0 = int(blockIdx.y) * per, g1 = min(p.G, g0 + per);
  const int l = lane_id(), w = wave_id(), half = l >> 5;
  const int wm = (w % WM) * (BM / WM), wn = (w / WM) * (BN / WN);
  // Rows past the matrix repeat its last one: what they give is not stored.  Offsets from
  // the tile's first row: at most 256 rows of 2^30 bytes.
  const uint8_t *ga = p.a + int64_t(m0) * p.K, *gb = p.b + int64_t(n0) * p.K;
  typedef typename Off<DMA>::T off_t;
  off_t pa[LA], pb[LB];
  // load i of the wave fills rows 8 i .. + 7 of its part; lane l its piece l mod 8 of row l / 8
  static_assert(LA % 2 == 0 && LB % 2 == 0, "rows of load i: i mod 2 decides their places");
  const int piece = (l & 7) ^ (l >> 4);   // for even i; ^ 4 for odd i
#pragma unroll
  for (int i = 0; i < LA; ++i) pa[i] = off_t(min((w * LA + i) * 8 + (l >> 3), p.M - 1 - m0)) * off_t(p.K);
#pragma unroll
  for (int i = 0; i < LB; ++i) pb[i] = off_t(min((w * LB + i) * 8 + (l >> 3), p.N - 1 - n0)) * off_t(p.K);
  u32x4 ra[DMA ? 1 : LA], rb[DMA ? 1 : LB];
  auto load = [&](int g, int buf) {
    const int k[2] = {g * kGroup + 16 * piece, g * kGroup + 16 * (piece ^ 4)};
    if constexpr (DMA) {
      if ((g + 1) * kGroup <= p.K) {
#pragma unroll
        for (int i = 0; i < LA; ++i) dma16(ga + pa[i] + k[i & 1], as[buf] + (w * LA + i) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i) dma16(gb + pb[i] + k[i & 1], bs[buf] + (w * LB + i) * 1024);
      } else {   // whole pieces, or zeros past the row's end
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < LA; ++i) {
          if (k[i & 1] < p.K) dma16(ga + pa[i] + k[i & 1], as[buf] + (w * LA + i) * 1024);
          else *reinterpret_cast<u32x4*>(as[buf] + (w * LA + i) * 1024 + 16 * l) = none;
        }
#pragma unroll
        for (int i = 0; i < LB; ++i) {
          if (k[i & 1] < p.K) dma16(gb + pb[i] + k[i & 1], bs[buf] + (w * LB + i) * 1024);
          else *reinterpret_cast<u32x4*>(bs[buf] + (w * LB + i) * 1024 + 16 * l) = none;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < LA; ++i) ra[i] = bytes16(ga + pa[i] + k[i & 1], p.K - k[i & 1]);
#pragma unroll
      for (int i = 0; i < LB; ++i) rb[i] = bytes16(gb + pb[i] + k[i & 1], p.K - k[i & 1]);
    }
  };
  auto put_tiles = [&](int buf) {
    if constexpr (!DMA) {
#pragma unroll
      for (int i = 0; i < LA; ++i) *reinterpret_cast<u32x4*>(as[buf] + (w * LA + i) * 1024 + 16 * l) = ra[i];
#pragma unroll
      for (int i = 0; i < LB; ++i) *reinterpret_cast<u32x4*>(bs[buf] + (w * LB + i) * 1024 + 16 * l) = rb[i];
    }
  };
  const float* psc[SC];
#pragma unroll
  for (int i = 0; i < SC; ++i) {
    const int t = i * NT + threadIdx.x;
    psc[i] = t < BM ? p.sa + int64_t(min(m0 + t, p.M - 1)) * p.G
                    : p.sb + int64_t(min(n0 + t - BM, p.N - 1) / (ROWS ? 1 : kGroup)) * p.G;
  }
  float rs[SC];
  auto load_scales = [&](int g) {
#pragma unroll
    for (int i = 0; i < SC; ++i)
      if (i * NT + int(threadIdx.x) < BM + BN) rs[i] = psc[i][g];
  };
  auto put_scales = [&](int buf) {
#pragma unroll
    for (int i = 0; i < SC; ++i)
      if (i * NT + int(threadIdx.x) < BM + BN) ss[buf][i * NT + threadIdx.x] = rs[i];
  };
  f32x16 acc[QT][MT];
#pragma unroll
  for (int j = 0; j < QT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
  // Row i of the instruction is row 16 (i / 4 % 2) + 4 (i / 8) + i % 4 of the 32: a lane's
  // 16 sums then belong to 16 neighbours
  const int li = l & 31, br = 16 * ((li >> 2) & 1) + 4 * (li >> 3) + (li & 3);
  if (g0 < g1) {
    load_scales(g0);
    load(g0, 0);
    put_scales(0);
    put_tiles(0);
  }
  for (int g = g0; g < g1; ++g) {
    const int buf = (g - g0) & 1;
    wait_vm<0>();
    chain_barrier();
    const bool more = g + 1 < g1;
    if (more) {
      load_scales(g + 1);
      load(g + 1, buf ^ 1);
    }
    typename Bytes<EXACT>::T fa[MT][2];
    float sa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) fa[i][kk] = operand<EXACT>(frag(as[buf], wm + 32 * i + li, kk));
      sa[i] = ss[buf][wm + 32 * i + li];
      if constexpr (!ROWS) sa[i] *= ss[buf][BM + wn];   // the wave's rows of b lie in one block of 128
    }
    // The sums of one tile are scaled while the next one's are formed
    typename Bytes<EXACT>::T fb[2];
    f32x16 x[2];
    auto scale_in = [&](int t) {
      const int j = t / MT, i = t % MT;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float s = ROWS ? sa[i] * ss[buf][BM + wn + 32 * j + 16 * half + r] : sa[i];
        acc[j][i][r] = fmaf(x[t & 1][r], s, acc[j][i][r]);
      }
      // the compiler would otherwise put all of these behind the loop's last branch and keep
      // every tile's sums until then
      asm volatile("" : "+v"(acc[j][i]));
    };
#pragma unroll
    for (int t = 0; t < QT * MT; ++t) {
      const int j = t / MT, i = t % MT;
      if (i == 0) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) fb[kk] = operand<EXACT>(frag(bs[buf], wn + 32 * j + br, kk));
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) x[t & 1][r] = 0.f;
      x[t & 1] = mul32(fb[0], fa[i][0], x[t & 1]);
      x[t & 1] = mul32(fb[1], fa[i][1], x[t & 1]);
      __builtin_amdgcn_sched_barrier(0);   // the next tile's instructions go first, then the scaling in their shadow
      if (t) scale_in(t - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    scale_in(QT * MT - 1);
    if (more) {
      put_scales(buf ^ 1);
      put_tiles(buf ^ 1);
    }
  }
  void* c = p.plan.splits > 1 ? static_cast<void*>(p.part + int64_t(blockIdx.y) * p.M * p.N) : p.c;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + wm + 32 * i + li;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      const int n = n0 + wn + 32 * j + 16 * half;
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = acc[j][i][r];
      put<T, 16>(c, int64_t(m) * p.N + n, p.N - n, x);
    }
  }
}

// The sum of the runs of a split contraction, in their order
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_sum(const GemmParams p) {
  const int64_t e = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4, all = int64_t(p.M) * p.N;
  if (e >= all) return;
  const int n = int(min(int64_t(4), all - e));
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.plan.splits; ++s) {
    const float* q = p.part + s * all + e;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) x[i] += q[i];
  }
  T* d = static_cast<T*>(p.c) + e;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) d[i] = T(x[i]);
}

// ---------------------------------------------------------------------------
// few rows of a
// ---------------------------------------------------------------------------
// A workgroup of 8 waves takes 16 rows of b and all of a's, its waves every eighth group
// of the contraction each (32 bytes of a lane's row straight from memory: every byte of b
// is used once), and adds their sums in LDS.  Bound by the bytes of b.
constexpr int kFewWaves = 8;

template <typename T, int MT, bool ROWS>
__global__ __launch_bounds__(64 * kFewWaves) void k_gemm_few(const GemmParams p) {
  constexpr int U = 2;   // groups a wave has on their way
  __shared__ __attribute__((aligned(16))) float sum[kFewWaves][16 * MT][20];   // [row of a][row of b], padded
  const int l = lane_id(), w = wave_id(), q = l & 15, h = l >> 4;
  const int n0 = int(blockIdx.x) * 16;
  const uint8_t* pb = p.b + int64_t(min(n0 + q, p.N - 1)) * p.K + 32 * h;
  const uint8_t* pa[MT];
  const float *psa[MT], *psb[ROWS ? 4 : 1];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min(16 * i + q, p.M - 1);
    pa[i] = p.a + m * p.K + 32 * h;
    psa[i] = p.sa + m * p.G;
  }
#pragma unroll
  for (int r = 0; r < (ROWS ? 4 : 1); ++r) psb[r] = p.sb + int64_t(ROWS ? min(n0 + 4 * h + r, p.N - 1) : n0 / kGroup) * p.G;
  auto bytes32 = [&](const uint8_t* s, int g) {
    const int k = g * kGroup, n = p.K - k - 32 * h;
    u32x4 lo, hi;
    lo = bytes16(s + k, n);
    hi = bytes16(s + k + 16, n - 16);
    return __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = zero4();
  for (int g0 = w; g0 < p.G; g0 += kFewWaves * U) {
    i32x8 fb[U], fa[U][MT];
    float sa[U][MT], sb[U][ROWS ? 4 : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * kFewWaves;
      if (g >= p.G) continue;
      fb[u] = bytes32(pb, g);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fa[u][i] = bytes32(pa[i], g);
        sa[u][i] = psa[i][g];
      }
#pragma unroll
      for (int r = 0; r < (ROWS ? 4 : 1); ++r) sb[u][r] = psb[r][g];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g0 + u * kFewWaves >= p.G) continue;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const f32x4 x = mul16(operand<sizeof(T) == 4>(fb[u]), operand<sizeof(T) == 4>(fa[u][i]), zero4());
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = fmaf(x[r], sa[u][i] * sb[u][ROWS ? r : 0], acc[i][r]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) *reinterpret_cast<f32x4*>(&sum[w][16 * i + q][4 * h]) = acc[i];
  __syncthreads();
  if (threadIdx.x >= 64 * MT) return;
  const int m = threadIdx.x >> 2, c = 4 * (threadIdx.x & 3);
  f32x4 s = *reinterpret_cast<const f32x4*>(&sum[0][m][c]);
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) {
    const f32x4 y = *reinterpret_cast<const f32x4*>(&sum[i][m][c]);
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] += y[r];
  }
  if (m >= p.M) return;
  T* d = static_cast<T*>(p.c) + int64_t(m) * p.N + n0 + c;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (n0 + c + r < p.N) d[r] = T(s[r]);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename T, bool ROWS>
int few(const GemmParams& p, hipStream_t s) {
  const unsigned grid = unsigned((p.N + 15) / 16);
  if (p.M <= 16) k_gemm_few<T, 1, ROWS><<<grid, 64 * kFewWaves, 0, s>>>(p);
  else if (p.M <= 32) k_gemm_few<T, 2, ROWS><<<grid, 64 * kFewWaves, 0, s>>>(p);
  else k_gemm_few<T, 4, ROWS><<<grid, 64 * kFewWaves, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool EXACT, bool ROWS>
int tiles(const GemmParams& p, hipStream_t s) {
  const bool dma = p.K % 16 == 0 && p.K <= (1 << 24);   // 128 rows within 32 bits
  if (p.plan.kind == 2) {
    const dim3 grid(unsigned(((p.M + 255) / 256) * ((p.N + 255) / 256)), unsigned(p.plan.splits));
    if constexpr (sizeof(T) == 2) k_gemm<T, 256, 256, 4, 2, false, ROWS, true><<<grid, 512, 0, s>>>(p);
  } else {
    const dim3 grid(unsigned(((p.M + 127) / 128) * ((p.N + 127) / 128)), unsigned(p.plan.splits));
    if (dma) k_gemm<T, 128, 128, 2, 2, EXACT, ROWS, true><<<grid, 256, 0, s>>>(p);
    else k_gemm<T, 128, 128, 2, 2, EXACT, ROWS, false><<<grid, 256, 0, s>>>(p);
  }
  return static_cast<int>(hipGetLastError());
}

template <typename T>
int launch_type(const GemmParams& p, hipStream_t s) {
  constexpr bool exact = sizeof(T) == 4;
  const bool rows = p.block == 1;
  if (p.plan.kind == 0) return rows ? few<T, true>(p, s) : few<T, false>(p, s);
  if (p.plan.splits == 1) return rows ? tiles<T, exact, true>(p, s) : tiles<T, exact, false>(p, s);
  if (const int e = rows ? tiles<float, exact, true>(p, s) : tiles<float, exact, false>(p, s)) return e;
  k_gemm_sum<T><<<unsigned((int64_t(p.M) * p.N + 1023) / 1024), 256, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_gemm(const GemmParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.M == 0 || p.N == 0) return 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return p.dtype == GDR_BF16 ? launch_type<bf16>(p, s) : launch_type<float>(p, s);
}

}  // namespace gdr
