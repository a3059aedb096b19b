// Product of e4m3 matrices with a scale for each 128 of the contraction (gdr_gemm).
//
//   c[m][n] = sum_g sa[m][g] sb[n][g] sum_{k in g} a[m][k] b[n][k]
// The inner sum over a group's 128 elements is matrix instructions alone (one 16x16x128 of
// e4m3, or four 16x16x32 of bf16 where c is fp32), started from zero; what they leave is
// scaled and added in fp32, so that the scales need not be powers of two.  One product,
// sa sb, scales all 128 elements' sum: the two one after the other would double what the
// VALU does beside the matrix instructions (41 % of the cycles of large products).  Both
// scales may be as large or small as fp32 has them, as long as sa sb is a normal number.
// b's rows are the instruction's rows and a's its columns: a lane then holds sums of one row of a, whose scale
// is one register, and b's scale is the same for all of them where it belongs to a block of
// 128 rows.
//
// Large products are bound by matrix instructions and scaling in turn: the first take 55 % of
// the cycles and the VALU 41 %, hardly any of them together (32768 x 4096 x 4096: 485 to 550
// us by card = 2,000 to 2,270 TFLOP/s; its instructions alone, fed from registers, 365 to
// 380), ordinary ones by how far tiles fill 256 compute
// units and LDS feeds them (1000 x 2050 x 4100, fp32: 44 us; 2048 cubed, bf16: 15.3), small
// ones by latency (64 x 4096 x 4096: 12.8 us, of which the kernel 9.7; one row, 4096 x 2048:
// 6.8, of which the kernel 3.8).  One form spills, 6 registers: fp32 results, 128 x 128, block
// 1, rows through registers.
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "../gdr_lds.h"
#include "gdr_gemm.h"
#include "gdr_wide.h"

namespace gdr {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t __attribute__((ext_vector_type(4), aligned(1))) u32x4u;

// Sum over a group, 16 x 16: lane l's 32 bytes (piece l / 16 of a group) of row l mod 16.
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
__device__ __forceinline__ f32x4 mul16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mul16(const Bytes<true>::T& a, const Bytes<true>::T& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mma(a.v[i], b.v[i], c);
  return c;
}

// n of the 16 bytes at p, the rest zero; the matrix ends at `end`.  Only at its end are
// they taken one by one: elsewhere what follows a row is the next one, and is masked.
__device__ __forceinline__ u32x4 bytes16(const uint8_t* p, int n, const uint8_t* end) {
  u32x4 v = {0, 0, 0, 0};
  if (n <= 0) return v;
  if (p + 16 <= end) {
    v = *reinterpret_cast<const u32x4u*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = n - 4 * i;
      v[i] = k >= 4 ? v[i] : k <= 0 ? 0u : v[i] & ((1u << (8 * k)) - 1u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) v[i / 4] |= uint32_t(p[i]) << (8 * (i % 4));
  }
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
// LDS rows of 128 bytes, a group each; piece p (16 bytes) of a row at piece p ^ f.  A
// 16-byte read serves lanes 0-3, 12-15, 20-23 and 24-27 together (and three sets like it),
// which are 4 runs of 4 rows, two of them 2 pieces further on; banks are 256 bytes, two
// rows.  No two of a set meet where f is bit 1 of the row and, above it, minus the run's
// number.  Row m of a's 16 is row m of the tile (run m / 4); row m of b's 16 is row
// 16 (m / 4) + 4 t + m % 4 of 64 for the tile's t-th 16 (run: the row's 16), so that the
// sums of four of them are 16 neighbours of c in a lane.
__device__ __forceinline__ int turn_a(int r) { return ((r >> 1) & 1) | ((-(r >> 2) & 3) << 1); }
__device__ __forceinline__ int turn_b(int r) { return ((r >> 1) & 1) | ((-(r >> 4) & 3) << 1); }
__device__ __forceinline__ i32x8 frag(const char* row, int f) {
  const int p = 2 * (lane_id() >> 4);
  const u32x4 lo = *reinterpret_cast<const u32x4*>(row + ((p ^ f) << 4));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(row + (((p + 1) ^ f) << 4));
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

// 16 bytes a lane from p + lane_off + wave_off to lds + 16 lane.  The buffer's size is no
// check here: callers stay within the matrix.
__device__ __forceinline__ void copy16(const uint8_t* p, uint32_t lane_off, int wave_off, char* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7fffffff, 0x00027000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)((lds_char_t*)lds), 16, lane_off, wave_off, 0, 0);
}

template <bool SHORT> struct Off { typedef uint32_t T; };
template <> struct Off<false> { typedef int64_t T; };

// T: what the sums are stored as (fp32 for the partial sums of a split contraction).
// NB: groups in LDS.  ROWS: b has a scale for each row.  DMA: rows start on 4 bytes,
// as loads to LDS ask for.
template <typename T, int BM, int BN, int WM, int WN, int NB, bool EXACT, bool ROWS, bool DMA>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_gemm(const GemmParams p) {
  constexpr int NT = 64 * WM * WN, MT = BM / WM / 16, QT = BN / WN / 16;
  constexpr int LA = BM / 8 / (WM * WN), LB = BN / 8 / (WM * WN);   // 1 KB loads a wave
  static_assert(QT % 4 == 0 && BM + BN <= NT && (DMA || NB == 2), "");
  constexpr int LOADS = LA + LB + 1;                                // of a wave and group, its scales included
  constexpr int PER = (LA + LB + QT - 3) / (QT == 4 ? 2 : QT - 2);   // tiles' loads with each tile of 16 rows of b
  __shared__ __attribute__((aligned(1024))) char as[NB][BM * 128], bs[NB][BN * 128];
  __shared__ __attribute__((aligned(16))) float ss[NB][NT];
  int tm, tn;
  tile_at(int(blockIdx.x), (p.M + BM - 1) / BM, (p.N + BN - 1) / BN, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  const int per = (p.G + p.plan.splits - 1) / p.plan.splits, g0 = int(blockIdx.y) * per, g1 = min(p.G, g0 + per);
  const int l = lane_id(), w = __builtin_amdgcn_readfirstlane(wave_id()), h = l >> 4, li = l & 15;
  const int wm = (w % WM) * (BM / WM), wn = (w / WM) * (BN / WN);
  // Load i of a wave fills rows 8 (w L + i) + l / 8, lane l the place l mod 8.  Rows past the
  // matrix repeat its last one: what they give is not stored.  Offsets from the tile's first
  // row: at most 256 rows of 2^22 bytes.
  const uint8_t *ga = p.a + int64_t(m0) * p.K, *gb = p.b + int64_t(n0) * p.K;
  typedef typename Off<DMA>::T off_t;
  off_t at[LA + LB];
  auto row_of = [&](int u) { return (u < LA ? w * LA + u : w * LB + u - LA) * 8 + (l >> 3); };
  auto piece_of = [&](int u) { return (l & 7) ^ (u < LA ? turn_a(row_of(u)) : turn_b(row_of(u))); };
#pragma unroll
  for (int u = 0; u < LA + LB; ++u)
    at[u] = off_t(min(row_of(u), u < LA ? p.M - 1 - m0 : p.N - 1 - n0)) * off_t(p.K) + off_t(16 * piece_of(u));
  auto spot = [&](int u, int buf) { return u < LA ? as[buf] + (w * LA + u) * 1024 : bs[buf] + (w * LB + u - LA) * 1024; };
  u32x4 raw[DMA ? 1 : LA + LB];
  // load u of a whole group g
  auto load = [&](int u, int g, int buf) {
    if constexpr (DMA)
      copy16(u < LA ? ga : gb, at[u], g * kGroup, spot(u, buf));
    else
      raw[u] = *reinterpret_cast<const u32x4u*>((u < LA ? ga : gb) + int64_t(g) * kGroup + at[u]);
  };
  // all of a last group that is shorter: zeros past the row's end
  auto load_tail = [&](int g, int buf) {
#pragma unroll
    for (int u = 0; u < LA + LB; ++u) {
      const uint8_t* src = (u < LA ? ga : gb) + int64_t(g) * kGroup + at[u];
      const int n = p.K - g * kGroup - 16 * piece_of(u);
      const u32x4 v = bytes16(src, n, u < LA ? p.a + int64_t(p.M) * p.K : p.b + int64_t(p.N) * p.K);
      if constexpr (DMA) *reinterpret_cast<u32x4*>(spot(u, buf) + 16 * l) = v;
      else raw[u] = v;
    }
  };
  auto put_tiles = [&](int buf) {
    if constexpr (!DMA) {
#pragma unroll
      for (int u = 0; u < LA + LB; ++u) *reinterpret_cast<u32x4*>(spot(u, buf) + 16 * l) = raw[u];
    }
  };
  // a thread's row of scales: of a, then of b
  const int t = threadIdx.x;
  const float* psc = t < BM ? p.sa + int64_t(min(m0 + t, p.M - 1)) * p.G
                            : p.sb + int64_t(min(n0 + min(t - BM, BN - 1), p.N - 1) / (ROWS ? 1 : kGroup)) * p.G;
  auto load_scale = [&](int g, int buf) { dma4(psc + g, reinterpret_cast<char*>(&ss[buf][64 * w])); };
  f32x4 acc[QT][MT];
#pragma unroll
  for (int j = 0; j < QT; ++j)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[j][i] = zero4();
  typedef typename Bytes<EXACT>::T Op;
  i32x8 fa[MT], fb[2];   // as they lie in LDS; EXACT turns them into bf16 when they are used
  float sa[MT];
  auto read_a = [&](int buf, int i) { return frag(as[buf] + (wm + 16 * i + li) * 128, turn_a(li)); };
  auto read_b = [&](int buf, int j) {
    const int r = 16 * (li >> 2) + (li & 3);
    return frag(bs[buf] + (wn + 64 * (j / 4) + 4 * (j % 4) + r) * 128, turn_b(r));
  };
  // the wave's rows of b lie in one block of 128
  auto read_scale = [&](int buf, int i) { return ss[buf][wm + 16 * i + li] * (ROWS ? 1.f : ss[buf][BM + wn]); };
  // the group after the one in use has come; the loads of later ones may be on their way
  auto publish = [&]() {
    wait_vm<(NB - 2) * LOADS>();
    chain_barrier();
  };
  // A last group that is shorter comes first, so that the loop loads whole groups alone.
  const int n = g1 - g0;
  const bool tail = g1 == p.G && p.K % kGroup != 0;
  auto group = [&](int i) { return tail ? (i == 0 ? g1 - 1 : g0 + i - 1) : g0 + i; };
  load_scale(group(0), 0);
  if (tail) {
    load_tail(g1 - 1, 0);
  } else {
#pragma unroll
    for (int u = 0; u < LA + LB; ++u) load(u, g0, 0);
  }
  put_tiles(0);
#pragma unroll
  for (int i = 1; i < NB - 1; ++i) {
    load_scale(group(min(i, n - 1)), i);
    if (n > 1 || !tail) {
#pragma unroll
      for (int u = 0; u < LA + LB; ++u) load(u, group(min(i, n - 1)), i);
    }
  }
  if (n == 1) wait_vm<0>();   // there may be fewer loads than publish counts
  publish();
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    fa[i] = read_a(0, i);
    sa[i] = read_scale(0, i);
  }
  fb[0] = read_b(0, 0);
  // The it-th group is in buffer it mod NB while the one NB - 1 further on is loaded into the
  // buffer that the last one has left, a few loads a tile of 16 rows of b: all at once would
  // hold up every wave until the memory pipeline has taken them.  The barrier that shows the
  // next group stands before the last tile, whose operands are in registers by then, and the
  // next group's first operands are read under it.  Past the end the last group is loaded
  // again, so that the loads on their way are always as many as publish counts.
  int buf = 0, spare = NB - 1;
  for (int it = 0; it < n; ++it) {
    const int next = buf + 1 == NB ? 0 : buf + 1, gn = group(min(it + NB - 1, n - 1));
    const bool more = n > 1 || !tail;   // but for a contraction of less than one group
    float sn[MT];
    f32x4 x[2][MT], sb[2];
    Op oa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) oa[i] = operand<EXACT>(fa[i]);
    load_scale(gn, spare);
    auto scale_in = [&](int j) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][i][r] = fmaf(x[j & 1][i][r], ROWS ? sa[i] * sb[j & 1][r] : sa[i], acc[j][i][r]);
        // the compiler would otherwise put these behind the loop's end and keep all sums until then
        asm volatile("" : "+v"(acc[j][i]));
      }
    };
#pragma unroll
    for (int j = 0; j < QT; ++j) {
      if (ROWS) sb[j & 1] = *reinterpret_cast<const f32x4*>(&ss[buf][BM + wn + 64 * (j / 4) + 16 * h + 4 * (j % 4)]);
      if (j < QT - 1) {
        fb[(j + 1) & 1] = read_b(buf, j + 1);
      } else {
        put_tiles(next);
        publish();
        fb[0] = read_b(next, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      const Op ob = operand<EXACT>(fb[j & 1]);
      if constexpr (EXACT) {   // chains of four, side by side
#pragma unroll
        for (int i = 0; i < MT; ++i) x[j & 1][i] = zero4();
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < MT; ++i) x[j & 1][i] = mma(ob.v[e], oa[i].v[e], x[j & 1][i]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if constexpr (!EXACT) x[j & 1][i] = mul16(ob, oa[i], zero4());
        if (j == QT - 1) {
          fa[i] = read_a(next, i);
          sn[i] = read_scale(next, i);
        }
      }
      if (j * PER < LA + LB && more) {
#pragma unroll
        for (int u = j * PER; u < min((j + 1) * PER, LA + LB); ++u) load(u, gn, spare);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (j) scale_in(j - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    scale_in(QT - 1);
#pragma unroll
    for (int i = 0; i < MT; ++i) sa[i] = sn[i];
    spare = buf;
    buf = next;
  }
  wait_vm<0>();   // no load may reach LDS that is another workgroup's by then
  void* c = p.plan.splits > 1 ? static_cast<void*>(p.part + int64_t(blockIdx.y) * p.M * p.N) : p.c;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + wm + 16 * i + li;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < QT; j += 4) {
      const int n = n0 + wn + 16 * j + 16 * h;
      float x[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = acc[j + r / 4][i][r % 4];
      put<T, 16>(c, int64_t(m) * p.N + n, p.N - n, x);
    }
  }
}

// The sum of the runs of a split contraction, in their order
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_sum(const GemmParams p) {
  const int64_t e = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8, all = int64_t(p.M) * p.N;
  if (e >= all) return;
  const int n = int(min(int64_t(8), all - e));
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.plan.splits; ++s) {
    const float* q = p.part + s * all + e;
    if (n == 8) {
      const u32x4 a = *reinterpret_cast<const Wide<float>::T*>(q), b = *reinterpret_cast<const Wide<float>::T*>(q + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] += __uint_as_float(a[i]);
        x[4 + i] += __uint_as_float(b[i]);
      }
    } else {
      for (int i = 0; i < n; ++i) x[i] += q[i];
    }
  }
  put<T, 8>(p.c, e, n, x);
}

// ---------------------------------------------------------------------------
// few rows of a
// ---------------------------------------------------------------------------
// A workgroup of 8 waves takes 16 rows of b and all of a's, its waves every eighth group
// of the contraction each (two pieces of a lane's row straight from memory: every byte of b
// is used once; both operands take the group's bytes in the same order, whatever it is), and
// adds their sums in LDS.  Bound by latency and the bytes of b: 1 x 4096 x 2048 in 3.8 us.
// At 32 rows of a it is still the shorter one (32 x 4096 x 4096: 10.2 us, tiles of 64 x 128
// in 4 runs 12.4), at 64 not (16.3 and 12.9).
constexpr int kFewWaves = 8;

template <typename T, int MT, bool ROWS>
__global__ __launch_bounds__(64 * kFewWaves) void k_gemm_few(const GemmParams p) {
  constexpr int U = 2;   // groups a wave has on their way
  __shared__ __attribute__((aligned(16))) float sum[kFewWaves][16 * MT][20];   // [row of a][row of b], padded
  const int l = lane_id(), w = wave_id(), q = l & 15, h = l >> 4;
  const int n0 = int(blockIdx.x) * 16;
  const uint8_t* pb = p.b + int64_t(min(n0 + q, p.N - 1)) * p.K + 16 * h;
  const uint8_t* pa[MT];
  const float *psa[MT], *psb[ROWS ? 4 : 1];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = min(16 * i + q, p.M - 1);
    pa[i] = p.a + m * p.K + 16 * h;
    psa[i] = p.sa + m * p.G;
  }
#pragma unroll
  for (int r = 0; r < (ROWS ? 4 : 1); ++r) psb[r] = p.sb + int64_t(ROWS ? min(n0 + 4 * h + r, p.N - 1) : n0 / kGroup) * p.G;
  auto bytes32 = [&](const uint8_t* s, int g, const uint8_t* end) {
    const int k = g * kGroup, n = p.K - k - 16 * h;
    u32x4 lo, hi;
    if ((g + 1) * kGroup <= p.K) {
      lo = *reinterpret_cast<const u32x4u*>(s + k);
      hi = *reinterpret_cast<const u32x4u*>(s + k + 64);
    } else {
      lo = bytes16(s + k, n, end);
      hi = bytes16(s + k + 64, n - 64, end);
    }
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
      fb[u] = bytes32(pb, g, p.b + int64_t(p.N) * p.K);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fa[u][i] = bytes32(pa[i], g, p.a + int64_t(p.M) * p.K);
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
  else k_gemm_few<T, 2, ROWS><<<grid, 64 * kFewWaves, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename T, int BM, int BN, int WM, int WN, int NB, bool EXACT, bool ROWS, bool DMA>
int tile(const GemmParams& p, hipStream_t s) {
  const dim3 grid(unsigned(((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN)), unsigned(p.plan.splits));
  k_gemm<T, BM, BN, WM, WN, NB, EXACT, ROWS, DMA><<<grid, 64 * WM * WN, 0, s>>>(p);
  return static_cast<int>(hipGetLastError());
}

template <typename T, bool EXACT, bool ROWS>
int tiles(const GemmParams& p, hipStream_t s) {
  // Small tiles: 8 waves hide more of their waits (512 x 4096 x 4096, bf16: 21.1 us, with 4 waves
  // 22.3; 200 x 300 x 2100: 10.6, 13.0), but turn more bytes into bf16 twice where that is done
  // (1000 x 2050 x 4100, fp32: 50.4, 46.2).
  constexpr int WM = EXACT ? 2 : 4;
  if (p.plan.kind == kGemmSmall)
    return p.plan.copy ? tile<T, 64, 128, WM, 2, 3, EXACT, ROWS, true>(p, s) : tile<T, 64, 128, WM, 2, 2, EXACT, ROWS, false>(p, s);
  if constexpr (sizeof(T) == 2)   // bf16 results, a contraction that is not split
    if (p.plan.kind == kGemmLarge) return tile<T, 256, 256, 4, 2, 2, EXACT, ROWS, true>(p, s);
  return p.plan.copy ? tile<T, 128, 128, 2, 2, 2, EXACT, ROWS, true>(p, s) : tile<T, 128, 128, 2, 2, 2, EXACT, ROWS, false>(p, s);
}

template <typename T>
int launch_type(const GemmParams& p, hipStream_t s) {
  constexpr bool exact = sizeof(T) == 4;
  const bool rows = p.block == 1;
  if (p.plan.kind == kGemmFew) return rows ? few<T, true>(p, s) : few<T, false>(p, s);
  if (p.plan.splits == 1) return rows ? tiles<T, exact, true>(p, s) : tiles<T, exact, false>(p, s);
  if (const int e = rows ? tiles<float, exact, true>(p, s) : tiles<float, exact, false>(p, s)) return e;
  k_gemm_sum<T><<<unsigned((int64_t(p.M) * p.N + 2047) / 2048), 256, 0, s>>>(p);
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
