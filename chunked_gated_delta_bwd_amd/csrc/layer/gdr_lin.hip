// Linear attention with a decay for each head (gdr_lin_fwd, gdr_lin_bwd, gdr_lin_step).
//
//   S_t = c S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t,  c = e^lambda
// In blocks of 64 tokens, i and j counted within the block, S the state before it:
//   o_i = scale (sum_{j <= i} c^(i-j) (q_i . k_j) v_j + c^(i+1) S q_i)
//   S' = c^n S + sum_j c^(n-1-j) v_j k_j^T
// The gradients have the same form with other tensors in the three places (x, y, z):
//   o:  (q, k, v)    dq: (dO, v, k) with S^T        forwards
//   dv: (k, q, dO)   dk: (v, dO, q) with the transposed state's gradient, backwards,
//   R' = c^n R + scale sum_i c^(i+1) dO_i q_i^T,  R being what the block's last token sees,
// so one kernel, k_lin_out, computes all four.
//
// Long sequences are cut into segments: k_lin_local forms what each adds to the state,
// k_lin_carry runs the states through them, and k_lin_out walks every segment from its
// state.  The state stays in registers, 16 columns of S^T a wave, so that a block's
// products read LDS alone; a workgroup walks one head, since a block's work (64 tokens, 6
// MFLOP a head of 128) is a turn of a few microseconds and heads are many.
//
// T = 32768, 16 heads of 128, bf16 (a tensor is 134 MB): k_lin_local 70 to 85 us (two
// tensors: 55 at the rate of a large copy), k_lin_carry 8, k_lin_out 133 to 155 for one
// output (four tensors: 110) and 253 to 305 for the gradients of k and v together (220, or
// 165 with what both read counted once).  Forward and backward move 2.55 GB in 655 us, 3.9
// TB/s or 80 % of a large copy's rate, where 1.48 GB would do with q, k and v read by both
// calls: k_lin_local reads k and v, and q and dO, once more (0.5), and the launch of dq reads
// v, k and dO apart from that of dk and dv (0.42).  That is the larger part of the distance to
// the floor; the rest is the chain of a turn, from LDS through the products to the next, with
// two waves a SIMD, which the state's registers and the two blocks in LDS (114 KB) allow
// (matrix cores 24 %, VALU 33 %, LDS 29 % of the cycles).  k_lin_out<bf16, 128> uses all 256
// vector registers; backwards it spills 8 of them and 25 scalar ones (into vector registers),
// forwards 19 scalar ones, with heads of 64 31 and 27; fp32 spills none.  Measured slower: four
// waves of 32 columns, and two workgroups of half the registers a compute unit.  k_lin_step:
// 250 rows, 32 heads of 128 (1.02 GB of states read and written): 186 to 190 us, 5.4 TB/s.
#include <hip/hip_runtime.h>

#include "../gdr_device.h"
#include "../gdr_lds.h"
#include "gdr_lin.h"

namespace gdr {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// fragments of a type: 16 bytes of each lane, KS elements of the contraction a step
// ---------------------------------------------------------------------------
// Lane l = 16 g + q.  Accumulators hold rows 4 g + r, column q (see gdr_device.h).
template <typename T> struct Lin;

template <> struct Lin<bf16> {
  typedef bf16x8 Frag;
  static constexpr int KS = 32;      // elements of the contraction per step
  static constexpr int E = 8;        // of them per lane
  template <int W> static __device__ __forceinline__ int off(int r, int c) { return soff<W, 0>(r, c); }
  template <int W> static __device__ __forceinline__ Frag rk(const char* t, int r0, int k0) {
    return frag_rk_s<W, 0>(t, r0, k0);
  }
  template <int W> static __device__ __forceinline__ Frag kc(const char* t, int c0, int k0) {
    return frag_kc_s<W, 0>(t, c0, k0);
  }
  // Of 32 columns in two tiles, column m of tile u is 8 (m / 4) + 4 u + m % 4, so that the
  // accumulators of both hold eight neighbours per lane, as a row's fragment does.  Both
  // tiles' addresses differ by 8 bytes (see gdr_lds.h for the exclusive or).
  template <int W> static __device__ __forceinline__ Frag pair(const char* t, int c0, int u, int k0) {
    const int l = lane_id(), q = l & 15, r = 8 * (l >> 4) + (q >> 2);
    auto at = [&](int row) { return t + k0 * (2 * W) + ((prow<W>(row) * (2 * W) + (((q & 3) ^ swz<W, 0>(row)) << 4)) ^ (2 * c0)) + 8 * u; };
    return tr_pair(at(r), at(r + 4));
  }
  // the accumulators' four rows of tile t
  static __device__ __forceinline__ int row(int t, int g) { return 32 * (t >> 1) + 8 * g + 4 * (t & 1); }
  static __device__ __forceinline__ void mul(Frag a, Frag b, f32x4& c) { c = mma(a, b, c); }
  static __device__ __forceinline__ Frag state(f32x4 a, f32x4 b) {
    const uint2 lo = pack4_bf16(a[0], a[1], a[2], a[3]), hi = pack4_bf16(b[0], b[1], b[2], b[3]);
    return __builtin_bit_cast(Frag, u32x4{lo.x, lo.y, hi.x, hi.y});
  }
  static __device__ __forceinline__ void store4(char* p, float a, float b, float c, float d) {
    // as a vector: a struct's copy would lose the name of its array (see k_lin_out)
    const uint2 v = pack4_bf16(a, b, c, d);
    *reinterpret_cast<u32x2*>(p) = u32x2{v.x, v.y};
  }
  static constexpr int B = 64;       // tokens per block
  // whether a lane of the wave holds an infinity or a NaN: times zero, they alone are not zero
  static __device__ __forceinline__ bool any_bad(const Frag (&f)[2]) {
    const Frag none = {};
    const f32x4 x = mma(f[1], none, mma(f[0], none, zero4()));
    return __any(!(x[0] + x[1] + (x[2] + x[3]) == 0.f));
  }
  // 1 where element e is an infinity or a NaN, 0 elsewhere; the fragment with a 0 in its place.
  // In integers: sixteen comparisons' masks would spill what the loop around them keeps.
  static __device__ __forceinline__ uint32_t bad(Frag f, int e) {
    const uint32_t u = __builtin_bit_cast(u32x4, f)[e / 2] >> (16 * (e & 1));
    return ((u & 0x7f80u) + 0x80u) >> 15;
  }
  static __device__ __forceinline__ Frag without(Frag f, int e, uint32_t bit) {
    u32x4 u = __builtin_bit_cast(u32x4, f);
    u[e / 2] &= ~((0u - bit) & (0xffffu << (16 * (e & 1))));
    return __builtin_bit_cast(Frag, u);
  }
};

template <> struct Lin<float> {
  typedef f32x4 Frag;
  static constexpr int KS = 16;
  static constexpr int E = 4;
  // Piece c / 4 (16 bytes) of row r at piece (c / 4) ^ (r % 16), r % 8 where a row has 8
  template <int W> static __device__ __forceinline__ int off(int r, int c) {
    return r * (4 * W) + (((c >> 2) ^ (r & (W >= 64 ? 15 : 7))) << 4) + ((c & 3) << 2);
  }
  template <int W> static __device__ __forceinline__ Frag rk(const char* t, int r0, int k0) {
    const int l = lane_id();
    return *reinterpret_cast<const Frag*>(t + off<W>(r0 + (l & 15), k0 + 4 * (l >> 4)));
  }
  template <int W> static __device__ __forceinline__ Frag pair(const char* t, int c0, int u, int k0) {
    return kc<W>(t, c0 + 16 * u, k0);
  }
  static __device__ __forceinline__ int row(int t, int g) { return 16 * t + 4 * g; }
  template <int W> static __device__ __forceinline__ Frag kc(const char* t, int c0, int k0) {
    const int l = lane_id();
    Frag f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float*>(t + off<W>(k0 + 4 * (l >> 4) + e, c0 + (l & 15)));
    return f;
  }
  static __device__ __forceinline__ void mul(Frag a, Frag b, f32x4& c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = mma_f32(a[e], b[e], c);
  }
  static __device__ __forceinline__ Frag state(f32x4 a, f32x4) { return a; }
  static __device__ __forceinline__ void store4(char* p, float a, float b, float c, float d) {
    *reinterpret_cast<f32x4*>(p) = f32x4{a, b, c, d};
  }
  static constexpr int B = 32;
  static __device__ __forceinline__ bool any_bad(const Frag (&f)[2]) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b |= ((__float_as_uint(f[0][i]) & 0x7f800000u) + 0x00800000u) | ((__float_as_uint(f[1][i]) & 0x7f800000u) + 0x00800000u);
    return __any(b >> 31);
  }
  static __device__ __forceinline__ uint32_t bad(Frag f, int e) {
    return ((__float_as_uint(f[e]) & 0x7f800000u) + 0x00800000u) >> 31;
  }
  static __device__ __forceinline__ Frag without(Frag f, int e, uint32_t bit) {
    f[e] = __uint_as_float(__float_as_uint(f[e]) & (bit - 1u));
    return f;
  }
};

// ---------------------------------------------------------------------------
// segments and decays
// ---------------------------------------------------------------------------
__device__ __forceinline__ LinSeg seg_at(const LinParams& p, int s) {
  if (p.dense_T < 0) return p.tab[s];
  LinSeg r;
  r.nseg = p.dense_nseg;
  r.seq = s / r.nseg;
  r.idx = s % r.nseg;
  r.t0 = r.seq * p.dense_T + r.idx * p.seg;
  r.len = min(p.seg, p.dense_T - r.idx * p.seg);
  return r;
}

// Segment and head of a workgroup: the heads of a segment one after the other, since their
// rows lie side by side (T = 32768, 16 heads of 128, training: 718 us, and 733 with the
// segments of a head one after the other).  Value heads that share q and k go to one XCD
// (see chunk_head_at).
__device__ __forceinline__ void place_of(const LinParams& p, int id, int& c, int& h) {
  if (p.G > 1) {
    chunk_head_at(p, id, c, h);
  } else {
    c = id / p.H;
    h = id % p.H;
  }
}

// lambda in base-2 units.  A log decay of -inf counts as -1e30: c^0 is 1 and any other
// power 0, where -inf would make c^0 a NaN.
__device__ __forceinline__ float decay2(const LinParams& p, int h) {
  const float l = p.log_decay[h] * kLog2e;
  return l < -1e30f ? -1e30f : l;
}
// A state's decay by c^n.  Over one half it is S + (c^n - 1) S, so that a slow decay's rounding
// does not add up over the blocks of a long sequence; below, c^n - 1 would lose c^n's bits.
struct Decay {
  float f;
  uint32_t keep;   // all bits, or none
  __device__ __forceinline__ float operator()(float s) const { return fmaf(f, s, __uint_as_float(__float_as_uint(s) & keep)); }
};
__device__ __forceinline__ Decay decay_of(float l2, int n) {
  const float x = float(n) * l2;
  const bool slow = x > -1.f;
  return {slow ? expm1f(x * 0.6931471805599453f) : exp2f(x), slow ? ~0u : 0u};
}
// of one token; rounded to fp32, a decay of 1 - 1e-6 would be one of 1 - 1.013e-6
__device__ __forceinline__ Decay decay_of(float lambda) {
  const bool slow = lambda > -0.6931472f;
  return {slow ? expm1f(lambda) : expf(lambda), slow ? ~0u : 0u};
}

// Copies blocks of a tensor to LDS, by the D / 16 waves of a workgroup.  A lane's row and place
// in a load of 1 KB, and the piece that belongs there, are the same in each of its loads.
template <typename T, int D>
struct Mover {
  static constexpr int NW = D / 16, ROW = D * int(sizeof(T)), PR = ROW / 16, RPL = 1024 / ROW;   // pieces a row, rows a load
  static constexpr int TB = Lin<T>::B * ROW, LPT = TB / 1024 / NW;                                // a wave's loads of a tile
  static_assert(LPT >= 1 && TB / 1024 % NW == 0 && (NW * RPL) % 16 == 0, "the rows of a wave's loads turn alike");
  int w, row, piece;
  __device__ __forceinline__ explicit Mover(int wave) : w(wave) {
    row = w * RPL + lane_id() / PR;
    piece = (Lin<T>::template off<D>(row & 15, 0) % ROW / 16) ^ (lane_id() % PR);
  }
  // n rows from src on.  The buffer ends behind the last: no lane reads past it.  What those
  // lanes leave in LDS is for clear().
  __device__ __forceinline__ void operator()(const char* src, uint32_t pitch, int n, char* tile) const {
    const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(src), 0, int(uint32_t(n - 1) * pitch + ROW), 0x00027000);
#pragma unroll
    for (int a = 0; a < LPT; ++a)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void_t*)((lds_char_t*)(tile + (a * NW + w) * 1024)), 16,
                                               (a * NW * RPL + row) * pitch + 16 * piece, 0, 0, 0);
  }
  // zeros in a tile's rows from n on, when the block has come
  static __device__ __forceinline__ void clear(char* tile, int n) {
    for (int a = threadIdx.x; a < (Lin<T>::B - n) * PR; a += NW * 64) *reinterpret_cast<u32x4*>(tile + n * ROW + 16 * a) = u32x4{0, 0, 0, 0};
  }
};

// ---------------------------------------------------------------------------
// the state of a wave: columns [slab, slab + 16) of S^T, all D rows
// ---------------------------------------------------------------------------
template <typename T, int D>
struct State {
  static constexpr int KT = D / 16, JS = Lin<T>::B / Lin<T>::KS;
  f32x4 s[KT];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int t = 0; t < KT; ++t) s[t] = zero4();
  }
  // memory holds [z channel][y channel], or the transpose
  __device__ __forceinline__ void load(const float* m, bool transposed, int slab) {
    const int l = lane_id(), g = l >> 4, v = slab + (l & 15);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int k = Lin<T>::row(t, g);
      if (!transposed) {
        s[t] = *reinterpret_cast<const f32x4*>(m + v * D + k);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) s[t][r] = m[(k + r) * D + v];
      }
    }
  }
  __device__ __forceinline__ void store(float* m, int slab) const {
    const int l = lane_id(), g = l >> 4, v = slab + (l & 15);
#pragma unroll
    for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(m + v * D + Lin<T>::row(t, g)) = s[t];
  }
  __device__ __forceinline__ void decay(const Decay& d) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] = d(s[t][r]);
  }
  // S^T += y^T (w z).  The weighted z of bf16 tensors is a sum of bf16 parts: three (24 bits of
  // significand, as fp32) for states that are returned or that another segment starts from,
  // two (2^-16 is left) for a state that only meets x within the segment and is rounded to bf16
  // there itself.  With one part its rounding would be as large as that one, and the outputs'
  // error against 64 bits 2.7e-3 in place of 2.35e-3 (1.66e-3 is their own rounding), for 3.5 %
  // of the time (T = 32768, 16 heads of 128, training: 768 us with one, 795 with two).
  typedef typename Lin<T>::Frag Frag;
  static __device__ __forceinline__ Frag weighted(Frag z, const float (&w)[Lin<T>::E], int part) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] *= w[e];
      return z;
    } else {
      float x[8];
      IO<bf16>::unpack8(__builtin_bit_cast(u32x4, z), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= w[e];
        if (part > 0) x[e] = lo_part(x[e]);
        if (part > 1) x[e] = lo_part(x[e]);
      }
      return Lin<T>::state(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
    }
  }
  // parts FROM .. TO - 1
  template <int FROM, int TO>
  __device__ __forceinline__ void add(const char* y, const Frag (&z)[JS], const float (&w)[JS][Lin<T>::E]) {
    constexpr int N = sizeof(T) == 4 ? 1 : TO - FROM;
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      Frag x[N];
#pragma unroll
      for (int a = 0; a < N; ++a) x[a] = weighted(z[js], w[js], FROM + a);
#pragma unroll
      for (int t = 0; t < KT; ++t) {
        const Frag f = Lin<T>::template pair<D>(y, 32 * (t >> 1), t & 1, js * Lin<T>::KS);
#pragma unroll
        for (int a = 0; a < N; ++a) Lin<T>::mul(f, x[a], s[t]);
      }
    }
  }
};

// Weights of a block's tokens in the state's update: c^(n-1-j), or c^(j+1) backwards
template <typename T, bool REV>
__device__ __forceinline__ void state_weights(float l2, int n, float scale, float (&w)[Lin<T>::B / Lin<T>::KS][Lin<T>::E]) {
  const int g = lane_id() >> 4;
#pragma unroll
  for (int js = 0; js < Lin<T>::B / Lin<T>::KS; ++js)
#pragma unroll
    for (int e = 0; e < Lin<T>::E; ++e) {
      const int j = js * Lin<T>::KS + Lin<T>::E * g + e;
      w[js][e] = j < n ? scale * fast_exp2(float(REV ? j + 1 : n - 1 - j) * l2) : 0.f;
    }
}

// ---------------------------------------------------------------------------
// tables
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_lin_table(const LinParams p, const LinBatch b) {
  for (int i = blockIdx.x; i < b.n; i += gridDim.x) {
    const int nseg = max(1, int((uint32_t(b.len[i]) + uint32_t(p.seg) - 1) / uint32_t(p.seg)));
    for (int s = threadIdx.x; s < nseg; s += 256) {
      LinSeg r;
      r.t0 = b.t0[i] + s * p.seg;
      r.len = min(p.seg, b.len[i] - s * p.seg);
      r.seq = b.seq0 + i;
      r.idx = s;
      r.nseg = nseg;
      p.tab[b.row0[i] + s] = r;
    }
    if (threadIdx.x == 0) {
      p.row0[b.seq0 + i] = b.row0[i];
      p.row0[b.seq0 + i + 1] = b.row0[i] + nseg;
    }
  }
}

// ---------------------------------------------------------------------------
// a segment's own contribution to the state after it (before it, backwards)
// ---------------------------------------------------------------------------
template <typename T, int D, bool REV>
__global__ __launch_bounds__(D * 4, 2) void k_lin_local(const LinParams p) {
  constexpr int kB = Lin<T>::B, JS = kB / Lin<T>::KS, TB = Mover<T, D>::TB, ROW = Mover<T, D>::ROW;
  __shared__ __attribute__((aligned(1024))) char tiles0[2][TB], tiles1[2][TB];   // apart, as in k_lin_out
  int c, h;
  place_of(p, int(blockIdx.x), c, h);
  const LinSeg sg = seg_at(p, c);
  if (REV ? sg.idx == 0 : sg.idx == sg.nseg - 1) return;   // nothing starts from it
  const float l2 = decay2(p, h);
  const int w = __builtin_amdgcn_readfirstlane(wave_id()), slab = w * 16, nb = (sg.len + kB - 1) / kB;
  const int n_last = sg.len - (nb - 1) * kB;
  auto rows = [&](int i) { return i == (REV ? 0 : nb - 1) ? n_last : kB; };   // of the walk's i-th block
  const Mover<T, D> mover(w);
  const int64_t t0 = sg.t0 + (REV ? (nb - 1) * kB : 0), step = REV ? -kB : kB;
  const uint32_t pitch[2] = {uint32_t(p.Hk) * ROW, uint32_t(p.H) * ROW};
  const char* src[2] = {static_cast<const char*>(REV ? p.q : p.k) + (t0 * p.Hk + h / p.G) * ROW,
                        static_cast<const char*>(REV ? p.dO : p.v) + (t0 * p.H + h) * ROW};
  auto load = [&](int i, auto& tiles, int m) {
    mover(src[m], pitch[m], rows(i), tiles[m]);
    src[m] += step * pitch[m];
  };
  load(0, tiles0, 0);
  load(0, tiles0, 1);
  State<T, D> S;
  S.zero();
  float wz[JS][Lin<T>::E];
  Decay over = {};   // a block
  int wn = -1;
  auto turn = [&](int i, auto& tiles, auto& next) {
    wait_vm<0>();
    chain_barrier();
    const int n = rows(i);
    if (n != wn) {
      state_weights<T, REV>(l2, n, REV ? p.scale : 1.f, wz);
      over = decay_of(l2, n);
      wn = n;
    }
    if (n < kB) {
      for (int m = 0; m < 2; ++m) mover.clear(tiles[m], n);
      chain_barrier();
    }
    typename Lin<T>::Frag zf[JS];
#pragma unroll
    for (int js = 0; js < JS; ++js) zf[js] = Lin<T>::template kc<D>(tiles[1], slab, js * Lin<T>::KS);
    if (i + 1 < nb) load(i + 1, next, 0);
    S.decay(over);
    if (i + 1 < nb) load(i + 1, next, 1);
    S.template add<0, 3>(tiles[0], zf, wz);
  };
  for (int i = 0; i < nb; i += 2) {
    turn(i, tiles0, tiles1);
    if (i + 1 < nb) turn(i + 1, tiles1, tiles0);
  }
  S.store((REV ? p.dst : p.st) + (int64_t(c) * p.H + h) * (D * D), slab);
}

// In place: from each segment's own contribution to the state that it starts from.
template <int D, bool REV>
__global__ __launch_bounds__(256) void k_lin_carry(const LinParams p) {
  constexpr int PER = D * D / 4 / 256;   // workgroups a state
  const int part = blockIdx.x % PER, h = blockIdx.x / PER % p.H, n = blockIdx.x / PER / p.H;
  int row0, nseg, len;                   // of the last segment
  if (p.dense_T < 0) {
    row0 = p.row0[n];
    nseg = p.row0[n + 1] - row0;
    len = p.tab[row0 + nseg - 1].len;
  } else {
    nseg = p.dense_nseg;
    row0 = n * nseg;
    len = p.dense_T - (nseg - 1) * p.seg;
  }
  if (nseg == 1) return;
  const float l2 = decay2(p, h);
  const int64_t e = 4 * (part * 256 + int(threadIdx.x)), step = int64_t(p.H) * D * D;
  const float* init = REV ? p.dht : p.h0;
  f32x4 cur = zero4();
  if (init) cur = *reinterpret_cast<const f32x4*>(init + (int64_t(n) * p.H + h) * (D * D) + e);
  float* st = (REV ? p.dst : p.st) + (int64_t(row0) * p.H + h) * (D * D) + e;
  const Decay whole = decay_of(l2, p.seg), short_one = decay_of(l2, len);
  constexpr int U = 8;                   // segments whose loads are on their way together
  for (int i0 = 0; i0 < nseg; i0 += U) {
    f32x4 x[U];
#pragma unroll
    for (int a = 0; a < U; ++a)
      if (i0 + a < nseg - 1) x[a] = *reinterpret_cast<const f32x4*>(st + (REV ? nseg - 1 - i0 - a : i0 + a) * step);
#pragma unroll
    for (int a = 0; a < U; ++a)
      if (i0 + a < nseg) {
        *reinterpret_cast<f32x4*>(st + (REV ? nseg - 1 - i0 - a : i0 + a) * step) = cur;
        if (i0 + a < nseg - 1) {
          const Decay d = REV && i0 + a == 0 ? short_one : whole;
#pragma unroll
          for (int r = 0; r < 4; ++r) cur[r] = d(cur[r]) + x[a][r];
        }
      }
  }
}

// ---------------------------------------------------------------------------
// outputs
// ---------------------------------------------------------------------------
// out from the tensors x, y, z
struct LinRole {
  const void *x, *y, *z;
  void* out;
  float* last;            // state after the last segment (before the first, backwards), or NULL
  const float* first;     // state of the whole sequence's start (end, backwards), or NULL
  const float* st;        // states of the segments
  int32_t xk, yk, zk;     // 1: the tensor has Hk heads, 0: H
  int32_t transposed;     // the state's memory is [y channel][z channel]
  float pair, inter, add; // factors of the pairs' product, of S x, of the state's update
  int32_t wide;           // out is fp32 (a value head's share of the gradient of a grouped q or k)
};
// One launch: n roles that walk the same way.  Two workgroups on one XCD, started together,
// take the two roles of a segment and head, so that much of what both read comes from HBM
// once (T = 32768, 16 heads of 128, dk and dv: 0.57 GB fetched of 0.81 GB read).
struct LinRoles {
  LinRole r[2];
  int32_t n;
};

// A wave holds 16 columns of S^T (channels of z) in registers.  The tiles of x, y and z are
// copied to LDS one block ahead.
template <typename T, int D, bool REV>
__global__ __launch_bounds__(D * 4, 2) void k_lin_out(const LinParams p, const LinRoles roles) {
  typedef typename Lin<T>::Frag Frag;
  constexpr int kB = Lin<T>::B, KS = Lin<T>::KS, JS = kB / KS, E = Lin<T>::E, TI = kB / 16;
  constexpr int NW = Mover<T, D>::NW, ROW = Mover<T, D>::ROW, TB = Mover<T, D>::TB;
  constexpr int NPAIR = TI * TI / NW > 0 ? TI * TI / NW : 1, JSTEP = NW / TI;   // a wave's tiles of pairs
  constexpr int PB = kB * kB * int(sizeof(T));
  // Arrays of their own, each named where it is used: of one array with two halves the
  // compiler takes it that a read may meet the loads on their way, and waits for them.
  __shared__ __attribute__((aligned(1024))) char tiles0[3][TB], tiles1[3][TB], pairs0[PB], pairs1[PB];
  int c, h, id = blockIdx.x, role = 0;
  const int places = p.NC * p.H;
  if (roles.n == 2) {
    const int whole = places & ~7;       // workgroups 8 apart share an XCD
    if (id < 2 * whole) {
      role = id >> 3 & 1;
      id = (id >> 4) * 8 + (id & 7);
    } else {
      role = id >= whole + places;
      id -= role ? places : whole;
    }
  }
  const LinRole o = roles.r[role];
  place_of(p, id, c, h);
  const LinSeg sg = seg_at(p, c);
  const int l = lane_id(), q = l & 15, g = l >> 4, w = __builtin_amdgcn_readfirstlane(wave_id());
  const int slab = w * 16, nb = (sg.len + kB - 1) / kB;
  const float l2 = decay2(p, h);
  const int64_t sh = int64_t(sg.seq) * p.H + h;
  const int n_last = sg.len - (nb - 1) * kB;
  auto rows = [&](int i) { return i == (REV ? 0 : nb - 1) ? n_last : kB; };   // of the walk's i-th block
  const Mover<T, D> mover(w);
  // Where the walk's next block begins, of x, y and z and of the output, and the bytes between rows
  const int64_t t0 = sg.t0 + (REV ? (nb - 1) * kB : 0);
  const int OB = o.wide ? 4 : int(sizeof(T));
  const char* src[3];
  uint32_t pitch[3];
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    const bool shared = m == 0 ? o.xk : m == 1 ? o.yk : o.zk;
    const int heads = shared ? p.Hk : p.H, head = shared ? h / p.G : h;
    src[m] = static_cast<const char*>(m == 0 ? o.x : m == 1 ? o.y : o.z) + (t0 * heads + head) * ROW;
    pitch[m] = uint32_t(heads) * ROW;
  }
  const uint32_t out_pitch = uint32_t(p.H) * D * OB;
  char* out = static_cast<char*>(o.out) + (t0 * p.H + h) * (D * OB);
  auto load = [&](int i, auto& tiles, int m) {
    mover(src[m], pitch[m], rows(i), tiles[m]);
    src[m] += (REV ? -int64_t(kB) : int64_t(kB)) * pitch[m];
  };
  if (nb) {
#pragma unroll
    for (int m = 0; m < 3; ++m) load(0, tiles0, m);
  }
  State<T, D> S;
  const bool start = REV ? sg.idx == sg.nseg - 1 : sg.idx == 0, end = REV ? sg.idx == 0 : sg.idx == sg.nseg - 1;
  const bool exact = end && o.last;
  if (!start) S.load(o.st + (int64_t(c) * p.H + h) * (D * D), o.transposed, slab);
  else if (o.first) S.load(o.first + sh * (D * D), o.transposed, slab);
  else S.zero();
  // The wave's tiles of pairs: tokens i of tile w % TI, tokens j of w / TI and every JSTEP-th
  // on, and the decay between them.  No two tokens are as far apart as the segment is long: a
  // growth may leave fp32 there, and times the zeros behind a block's end would be a NaN.
  const int it0 = w % TI, jt0 = w / TI, gap0 = 16 * (it0 - jt0) + q - 4 * g;
  float near[NPAIR][4];
#pragma unroll
  for (int a = 0; a < NPAIR; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = gap0 - (16 * a * JSTEP + r), n = REV ? -d : d;
      near[a][r] = n >= 0 && n < sg.len ? o.pair * fast_exp2(float(n) * l2) : 0.f;
    }
  // the pairs of later tokens are never written again
  for (int i = threadIdx.x; i < PB / 16; i += NW * 64) {
    *reinterpret_cast<u32x4*>(pairs0 + 16 * i) = u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(pairs1 + 16 * i) = u32x4{0, 0, 0, 0};
  }
  float wz[JS][E], far[TI];
  Decay over = {};   // a block
  int wn = -1;
  // here and not at the state's first use, where the compiler would wait for every load that
  // is on its way, in each turn of the loop
  wait_vm<0>();
  // A block's sums, its z and where its infinities and NaN begin, until its pairs are there
  f32x4 acc[TI];
  Frag zf[JS];
  bool odd = false;
  int bad_from = kB;
#pragma unroll
  for (int it = 0; it < TI; ++it) acc[it] = zero4();
#pragma unroll
  for (int js = 0; js < JS; ++js) zf[js] = Frag{};
  // The pairs' part of the walk's i-th block, and its output; block -1 has none
  auto finish = [&](int i, auto& ps) {
#pragma unroll
    for (int js = 0; js < JS; ++js)
#pragma unroll
      for (int it = 0; it < TI; ++it) {
        if (REV ? (js + 1) * KS <= 16 * it : js * KS >= 16 * (it + 1)) continue;
        Lin<T>::mul(zf[js], Lin<T>::template rk<kB>(ps, 16 * it, js * KS), acc[it]);
      }
    if (odd) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int from = __shfl(bad_from, 4 * g + r, 64);
#pragma unroll
        for (int it = 0; it < TI; ++it)
          if ((REV ? kB - 1 - (16 * it + q) : 16 * it + q) >= from) acc[it][r] = __builtin_nanf("");
      }
    }
    // The buffer ends behind the block's last token, and is empty for block -1: what would lie
    // further on is dropped.
    const __amdgpu_buffer_rsrc_t dst = __builtin_amdgcn_make_buffer_rsrc(out, 0, i < 0 ? 0 : int(uint32_t(rows(i) - 1) * out_pitch + D * OB), 0x00027000);
    const uint32_t at = uint32_t(q) * out_pitch + slab * OB;
    if (i >= 0) out += (REV ? -int64_t(kB) : int64_t(kB)) * out_pitch;
    if (sizeof(T) == 4 || o.wide) {
#pragma unroll
      for (int it = 0; it < TI; ++it)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[it]), dst, at + 16 * it * out_pitch + 16 * g, 0, 0);
    } else {
#pragma unroll
      for (int it = 0; it < TI; ++it) {
        const uint2 v = pack4_bf16(acc[it][0], acc[it][1], acc[it][2], acc[it][3]);
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{v.x, v.y}, dst, at + 16 * it * out_pitch + 8 * g, 0, 0);
      }
    }
  };
  // pairs of a block: P[i][j] = c^|i-j| (x_i . y_j)
  auto pairs = [&](auto& tiles, auto& ps) {
    const char *const xs = tiles[0], *const ys = tiles[1];
    if (jt0 >= TI) return;
    int gap = gap0;
    asm volatile("" : "+v"(gap));   // compared each time: the masks of all turns would spill
    Frag xf[D / KS];
#pragma unroll
    for (int ks = 0; ks < D / KS; ++ks) xf[ks] = Lin<T>::template rk<D>(xs, 16 * it0, ks * KS);
#pragma unroll
    for (int s = 0; s < NPAIR; ++s) {
      const int jt = jt0 + s * JSTEP;
      if (REV ? jt < it0 : jt > it0) continue;
      f32x4 a = zero4();
#pragma unroll
      for (int ks = 0; ks < D / KS; ++ks) Lin<T>::mul(Lin<T>::template rk<D>(ys, 16 * jt, ks * KS), xf[ks], a);
      // a later token's product counts nothing, whatever it is
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = gap - (16 * s * JSTEP + r);
        a[r] = (REV ? d <= 0 : d >= 0) ? a[r] * near[s][r] : 0.f;
      }
      Lin<T>::store4(ps + Lin<T>::template off<kB>(16 * it0 + q, 16 * jt + 4 * g), a[0], a[1], a[2], a[3]);
    }
  };
  // Of a SIMD's two waves one forms its pairs first and the other last, so that they meet LDS
  // and the matrix cores in turns; the loads of the next block are spread over the turn's end,
  // where fewer reads of LDS wait behind them.  T = 32768, 16 heads of 128, training: 801 us
  // with neither, 780 with the first, 755 with both.
  const bool early = w < NW / 2;
  auto turn = [&](int i, auto& tiles, auto& next, auto& ps, auto& ps_before) {
    // The block has come, and so have the pairs of the block before.
    wait_vm<0>();
    chain_barrier();
    const int n = rows(i);
    if (n != wn) {
      state_weights<T, REV>(l2, n, o.add, wz);
      over = decay_of(l2, n);
#pragma unroll
      for (int it = 0; it < TI; ++it) {
        const int m = REV ? n - 1 - (16 * it + q) : 16 * it + q + 1;
        far[it] = m >= 0 ? o.inter * fast_exp2(float(m) * l2) : 0.f;
      }
      wn = n;
    }
    if (n < kB) {
      for (int m = 0; m < 3; ++m) mover.clear(tiles[m], n);
      chain_barrier();
    }
    const char *const xs = tiles[0], *const ys = tiles[1], *const zs = tiles[2];
    if (early) pairs(tiles, ps);
    finish(i - 1, ps_before);
    if (i + 1 < nb) load(i + 1, next, 0);
#pragma unroll
    for (int js = 0; js < JS; ++js) zf[js] = Lin<T>::template kc<D>(zs, slab, js * KS);
    // Infinities and NaN in z: a zero pair times one would reach tokens before it, so the
    // products take zeros in their place, and what comes from that token on is NaN: bad_from, in
    // the order of the walk, for the lane's column.
    odd = Lin<T>::any_bad(zf);
    if (odd) {
      bad_from = kB;
#pragma unroll
      for (int js = 0; js < JS; ++js)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int j = js * KS + E * g + e;
          const uint32_t bit = Lin<T>::bad(zf[js], e);
          zf[js] = Lin<T>::without(zf[js], e, bit);
          bad_from = min(bad_from, (REV ? kB - 1 - j : j) | int((bit - 1u) & 1024u));
        }
      bad_from = min(bad_from, __shfl_xor(bad_from, 16, 64));
      bad_from = min(bad_from, __shfl_xor(bad_from, 32, 64));
    }
#pragma unroll
    for (int it = 0; it < TI; ++it) acc[it] = zero4();
#pragma unroll
    for (int ks = 0; ks < D / KS; ++ks) {
      const Frag a = Lin<T>::state(S.s[ks * KS / 16], S.s[ks * KS / 16 + (KS == 32)]);
#pragma unroll
      for (int it = 0; it < TI; ++it) Lin<T>::mul(a, Lin<T>::template rk<D>(xs, 16 * it, ks * KS), acc[it]);
    }
#pragma unroll
    for (int it = 0; it < TI; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[it][r] *= far[it];
    if (i + 1 < nb) load(i + 1, next, 1);
    S.decay(over);
    S.template add<0, 2>(ys, zf, wz);
    if (sizeof(T) == 2 && exact) S.template add<2, 3>(ys, zf, wz);
    if (i + 1 < nb) load(i + 1, next, 2);
    if (odd && bad_from < kB) {
#pragma unroll
      for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S.s[t][r] = __builtin_nanf("");
    }
    if (!early) pairs(tiles, ps);
  };
  for (int i = 0; i < nb; i += 2) {
    turn(i, tiles0, tiles1, pairs0, pairs1);
    if (i + 1 < nb) turn(i + 1, tiles1, tiles0, pairs1, pairs0);
  }
  if (nb) {
    chain_barrier();
    if (nb & 1) finish(nb - 1, pairs0);
    else finish(nb - 1, pairs1);
  }
  if (exact) S.store(o.last + sh * (D * D), slab);
}

// Sum of the G value heads' shares of a key head's gradient, in head order
template <typename T>
__global__ __launch_bounds__(256) void k_lin_group(const float* __restrict__ src, void* __restrict__ dst, int64_t n8,
                                                   int Hk, int D, int G) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n8) return;
  const int64_t e = i * 8, row = e / D;
  const int c = int(e - row * D);
  float acc[8], x[8];
  IO<float>::load8(src, row * G * D + c, acc);
  for (int m = 1; m < G; ++m) {
    IO<float>::load8(src, (row * G + m) * D + c, x);
#pragma unroll
    for (int a = 0; a < 8; ++a) acc[a] += x[a];
  }
  IO<T>::store8(dst, e, acc);
}

// ---------------------------------------------------------------------------
// single token
// ---------------------------------------------------------------------------
// Lane j of a row's eight holds channels 32 m + 4 j .. + 3 (see gdr_step.hip)
template <typename TIO, int D>
__device__ __forceinline__ void load_row(const void* base, int64_t off, int j, float (&x)[D / 8]) {
#pragma unroll
  for (int m = 0; m < D / 32; ++m) {
    float y[4];
    IO<TIO>::load4(base, off + 32 * m + 4 * j, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * m + e] = y[e];
  }
}

// One row of the state for every eight lanes, 32 rows a workgroup
template <typename T, int D>
__global__ __launch_bounds__(256) void k_lin_step(const LinStepParams p) {
  constexpr int E = D / 8, SPLIT = D / 32;
  const int64_t id = blockIdx.x;
  const int part = int(id % SPLIT);
  const int h = int(id / SPLIT % p.H);
  int n = int(id / SPLIT / p.H);
  const int slot = p.slots ? p.slots[n] : n;
  if (slot < 0 || slot >= p.P) return;
  const int j = threadIdx.x & 7, row = part * 32 + (threadIdx.x >> 3);
  float* st = p.state + (int64_t(slot) * p.H + h) * (D * D) + row * D;
  float S[E], q[E], k[E];
  load_row<float, D>(st, 0, j, S);
  load_row<T, D>(p.q, (int64_t(n) * p.Hk + h / p.G) * D, j, q);
  load_row<T, D>(p.k, (int64_t(n) * p.Hk + h / p.G) * D, j, k);
  float v = IO<T>::load1(p.v, (int64_t(n) * p.H + h) * D + row);
  const Decay a = decay_of(p.log_decay[h]);
  // the slot is another row's if an earlier one names it, and takes the later ones that do along
  bool later = false;
  if (p.slots) {
    bool earlier = false;
    for (int m = threadIdx.x; m < p.N; m += 256)
      if (p.slots[m] == slot) {
        earlier |= m < n;
        later |= m > n;
      }
    if (__syncthreads_or(earlier)) return;
    later = __syncthreads_or(later);
  }
  for (;;) {
    float o = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      S[e] = fmaf(v, k[e], a(S[e]));
      o = fmaf(S[e], q[e], o);
    }
    o = group_sum_dpp<8>(o);
    if (j == 0) IO<T>::store1(p.o, (int64_t(n) * p.H + h) * D + row, p.scale * o);
    if (!later) break;
    do ++n; while (n < p.N && p.slots[n] != slot);
    if (n >= p.N) break;
    load_row<T, D>(p.q, (int64_t(n) * p.Hk + h / p.G) * D, j, q);
    load_row<T, D>(p.k, (int64_t(n) * p.Hk + h / p.G) * D, j, k);
    v = IO<T>::load1(p.v, (int64_t(n) * p.H + h) * D + row);
  }
#pragma unroll
  for (int m = 0; m < D / 32; ++m) IO<float>::store4(st, 32 * m + 4 * j, S[4 * m], S[4 * m + 1], S[4 * m + 2], S[4 * m + 3]);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
int last_error() { return static_cast<int>(hipGetLastError()); }

template <typename T, int D>
int states(const LinParams& p, bool backward, hipStream_t s) {
  if (!p.split) return 0;
  const unsigned grid = unsigned(int64_t(p.NC) * p.H);
  if (backward) k_lin_local<T, D, true><<<grid, D * 4, 0, s>>>(p);
  else k_lin_local<T, D, false><<<grid, D * 4, 0, s>>>(p);
  if (const int e = last_error()) return e;
  const unsigned carry = unsigned(int64_t(p.N) * p.H * (D * D / 1024));
  if (backward) k_lin_carry<D, true><<<carry, 256, 0, s>>>(p);
  else k_lin_carry<D, false><<<carry, 256, 0, s>>>(p);
  return last_error();
}

template <typename T, int D, bool REV>
int out(const LinParams& p, const LinRoles& r, hipStream_t s) {
  k_lin_out<T, D, REV><<<unsigned(int64_t(p.NC) * p.H * r.n), D * 4, 0, s>>>(p, r);
  return last_error();
}

template <typename T, int D>
int fwd(const LinParams& p, hipStream_t s) {
  const LinRole o = {p.q, p.k, p.v, p.o, p.ht, p.h0, p.st, 1, 1, 0, 0, p.scale, p.scale, 1.f, 0};
  return out<T, D, false>(p, {{o, o}, 1}, s);
}

template <typename T, int D>
int bwd(const LinParams& p, hipStream_t s) {
  const int grouped = p.G > 1;
  const int64_t n8 = int64_t(p.T) * p.Hk * D / 8;
  auto sum = [&](void* dst) {
    if (grouped && n8) k_lin_group<T><<<unsigned((n8 + 255) / 256), 256, 0, s>>>(p.part, dst, n8, p.Hk, D, p.G);
    return last_error();
  };
  void* part = p.part;
  const LinRole q = {p.dO, p.v, p.k, grouped ? part : p.dq, nullptr, p.h0, p.st, 0, 0, 1, 1, p.scale, p.scale, 1.f, grouped};
  const LinRole k = {p.v, p.dO, p.q, grouped ? part : p.dk, nullptr, p.dht, p.dst, 0, 0, 1, 1, p.scale, 1.f, p.scale, grouped};
  const LinRole v = {p.k, p.q, p.dO, p.dv, p.dh0, p.dht, p.dst, 1, 1, 0, 0, p.scale, 1.f, p.scale, 0};
  if (const int e = out<T, D, false>(p, {{q, q}, 1}, s)) return e;
  if (const int e = sum(p.dq)) return e;
  if (const int e = out<T, D, true>(p, {{k, v}, 2}, s)) return e;
  return sum(p.dk);
}

template <typename T, int D>
int step(const LinStepParams& p, hipStream_t s) {
  k_lin_step<T, D><<<unsigned(int64_t(p.N) * p.H * (D / 32)), 256, 0, s>>>(p);
  return last_error();
}

#define GDR_LIN_DISPATCH(fn, ...)                                                              \
  (p.dtype == GDR_BF16 ? (p.D == 128 ? fn<bf16, 128>(__VA_ARGS__) : fn<bf16, 64>(__VA_ARGS__)) \
                       : (p.D == 128 ? fn<float, 128>(__VA_ARGS__) : fn<float, 64>(__VA_ARGS__)))

}  // namespace

int launch_lin_table(const LinParams& p, const LinBatch& b, void* stream) {
  (void)hipGetLastError();
  k_lin_table<<<unsigned(b.n), 256, 0, reinterpret_cast<hipStream_t>(stream)>>>(p, b);
  return last_error();
}

int launch_lin_states(const LinParams& p, bool backward, void* stream) {
  (void)hipGetLastError();
  if (p.NC == 0) return 0;
  return GDR_LIN_DISPATCH(states, p, backward, reinterpret_cast<hipStream_t>(stream));
}

int launch_lin_fwd(const LinParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.NC == 0) return 0;
  return GDR_LIN_DISPATCH(fwd, p, reinterpret_cast<hipStream_t>(stream));
}

int launch_lin_bwd(const LinParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.NC == 0) return 0;
  return GDR_LIN_DISPATCH(bwd, p, reinterpret_cast<hipStream_t>(stream));
}

int launch_lin_step(const LinStepParams& p, void* stream) {
  (void)hipGetLastError();
  if (p.N == 0) return 0;
  return GDR_LIN_DISPATCH(step, p, reinterpret_cast<hipStream_t>(stream));
}

}  // namespace gdr
