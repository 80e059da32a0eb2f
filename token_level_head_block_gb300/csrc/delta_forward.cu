// The gated delta rule, per (b, h):
//   S'_t = e^{g_t} S_{t-1},  w_t = beta_t (v_t - S'_t^T k_t),  S_t = S'_t + k_t w_t^T,  o_t = scale S_t^T q_t
// over chunks of C tokens.  With b_i the sum of the log decays of a chunk's tokens up to i, B that of all,
// D_ij = e^{b_i - b_j} and G = tril(K K^T . D, -1), the w of a chunk that S enters solve (1 + beta G) W = beta (V - e^b K S).
// So with T = (1 + beta G)^-1,
//   W = U - K^ S           U = T beta V,  K^ = T beta e^b K
//   O = scale (e^b Q S + tril(Q K^T . D) W)
//   S <- e^B S + (e^{B-b} K)^T W
// Only the first and the last line need S.  delta_prepare forms T, U, K^ and the scores of every chunk, all at once;
// delta_scan then walks a sequence's chunks.
//
// The scan is a chain of two products a chunk, so latency bounds it.  It runs transposed (S^T, W^T), a CTA with 16 or 32 columns of the
// state.  A warp of the chain forms the W of 16 tokens and then its share of the state's rows; W and the state pass between the
// warps as planes of fp16 pairs in shared memory, two barriers a chunk.  Two warps beside each of the chain's form its tokens' outputs
// from the same planes, half of the columns each; one of them fetches what all read with bulk copies, up to two chunks ahead.  What the scan
// reads lies as its fragments do, so that a lane takes 16 bytes of an operand at once.
//
// Measured, bf16 [4, 4096, 12, 64] and [4, 65536, 6, 64]:
//   delta_prepare  103 and 773 us, 92 KB read and written a chunk (42 and 340 us of HBM's time).  A chunk takes 25,000 cycles, three of
//     them on an SM at once: 4,000 until its rows are there, 5,000 for T's blocks, 4,500 in the products of K^ and U, the rest in gates,
//     scores and images; issue slots are 45% full, and the instruction cache misses one time in eight.  Scores formed while the other
//     warps invert took 111 us for 107; the rows of the CTA that follows asked for as far as L2, 141 for 132 (with the gradients' images).
//   delta_scan  107 and 1180 us: 96 CTAs of two tiles, 1.65 us a chunk, and 96 of one tile, 1.15 us.  With W and e^{B-b} W at one
//     scale the long scan took 1103, and the state lost its digits where a chunk fades; their two maxima through one pair of shuffles took
//     1190.  Before that, of 2,400 cycles a chunk (clocks read in between) 700 W's products, 400 its splitting, 550 the state's products, 450 its
//     splitting, 250 at the barriers; the chain alone, without outputs, 76 us for 105: the warps beside it share its issue slots and
//     tensor cores; one such warp for two 1142 us for 1103.  Asking L2 for a chunk's operands ahead of the copies took 1875 us for 1426.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "delta_common.cuh"
#include "tc_common.cuh"

namespace mhla {

__device__ unsigned int g_delta_error = 0;

using namespace delta;

namespace {

// A thread's share of one operand's rows, where they are 16-byte units: asked for together, before the first is waited for.
template <typename T, int DK, int THREADS>
struct Rows {
  static constexpr int C = Lay<T, DK>::C, E = 16 / sizeof(T), kUnits = C * DK / E, kEach = kUnits / THREADS;
  static_assert(kUnits % THREADS == 0, "whole passes");
  uint4 x[kEach];
  __device__ __forceinline__ void fetch(const T* src, int64_t sn, int rows, int d, bool wide) {
    if (!wide) return;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = threadIdx.x + THREADS * j, r = i / (DK / E), c = E * (i % (DK / E));
      x[j] = r < rows && c < d ? *reinterpret_cast<const uint4*>(src + r * sn + c) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

// Rows of one operand to planes of terms; zeros behind the last token and channel.
// WATCH 1: the first row with a value that is not finite to `first`; 2: each column's; such values are left as zeros.
// MOST: the largest size to *most.
template <typename T, int DK, int THREADS, int WATCH, bool MOST = (WATCH == 1)>
__device__ __forceinline__ void load_rows(char* dst, const Rows<T, DK, THREADS>& units, const T* src, int64_t sn, int rows, int d,
                                          bool wide, int32_t* first, uint32_t* most = nullptr) {
  float largest = 0.0f;
  using L = Lay<T, DK>;
  constexpr int C = L::C;
  auto watch = [&](float x, int r, int c) {
    if (WATCH != 0 && !finite(x)) {
      atomicMin(first + (WATCH == 2 ? c : 0), r);
      return 0.0f;
    }
    if (MOST) largest = fmaxf(largest, fabsf(x));
    return x;
  };
  if (wide) {
    using R = Rows<T, DK, THREADS>;
#pragma unroll
    for (int j = 0; j < R::kEach; ++j) {
      const int i = threadIdx.x + THREADS * j, r = i / (DK / R::E), c = R::E * (i % (DK / R::E));
      uint32_t w[4] = {units.x[j].x, units.x[j].y, units.x[j].z, units.x[j].w};
      if constexpr (sizeof(T) == 2) {
        if (WATCH != 0 || MOST) {
          uint32_t bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {   // 0 times what is not finite is NaN
            const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), __floats2bfloat162_rn(0.0f, 0.0f));
            bad |= *reinterpret_cast<const uint32_t*>(&z);
          }
          if (MOST || (bad & 0x7FFF7FFFu))
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack(watch(low(w[e]), r, c + 2 * e), watch(high(w[e]), r, c + 2 * e + 1));
        }
        *reinterpret_cast<uint4*>(dst + unit_at<DK>(r, c >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        uint32_t lo[L::kIn], hi[L::kIn];
        split<L::kIn>(watch(__uint_as_float(w[0]), r, c), watch(__uint_as_float(w[1]), r, c + 1), lo);
        split<L::kIn>(watch(__uint_as_float(w[2]), r, c + 2), watch(__uint_as_float(w[3]), r, c + 3), hi);
#pragma unroll
        for (int n = 0; n < L::kIn; ++n)
          *reinterpret_cast<uint2*>(dst + n * L::kRows + unit_at<DK>(r, c >> 3) + (c & 7) * 2) = make_uint2(lo[n], hi[n]);
      }
    }
  } else {
#pragma unroll 4
    for (int i = threadIdx.x; i < C * DK / 2; i += THREADS) {
      const int r = i / (DK / 2), c = 2 * (i % (DK / 2));
      const T* x = src + r * sn + c;
      const float a = r < rows && c < d ? watch(to_f(x[0]), r, c) : 0.0f;
      const float e = r < rows && c + 1 < d ? watch(to_f(x[1]), r, c + 1) : 0.0f;
      uint32_t t[L::kIn];
      split<L::kIn>(a, e, t);
#pragma unroll
      for (int n = 0; n < L::kIn; ++n)
        *reinterpret_cast<uint32_t*>(dst + n * L::kRows + unit_at<DK>(r, c >> 3) + (c & 7) * 2) = t[n];
    }
  }
  if (MOST) {
    const uint32_t all = __reduce_max_sync(~0u, __float_as_uint(largest));
    if ((threadIdx.x & 31) == 0) atomicMax(most, all);
  }
}

// A pair of values that planes of bf16 terms hold, scaled, as fp16.
template <int NI, int NH>
__device__ __forceinline__ void to_halves(const uint32_t (&x)[NI][4], int e, float by, uint32_t (&t)[NH]) {
  float a = low(x[NI - 1][e]), b = high(x[NI - 1][e]);
#pragma unroll
  for (int n = NI - 2; n >= 0; --n) {
    a += low(x[n][e]);
    b += high(x[n][e]);
  }
  halves<NH>(a * by, b * by, t);
}

template <typename T, int DK>
struct Prepare {
  using L = Lay<T, DK>;
  static constexpr int C = L::C, kStrips = L::kTiles, kThreads = 64 * kStrips;
  static constexpr int kPitch = C + 8;   // floats a row of T: a lane's pairs of eight rows meet all banks
  static constexpr int kK = (C * kPitch * 4 + 127) / 128 * 128, kV = kK + L::kInput, kQ = kV + L::kInput;
  // K^ on the way, float32: Q's place and what is behind it
  static constexpr int kKeep = kQ, kBytes = kQ + std::max(L::kInput, C * DK * 4);
};

// Planes of terms as planes of fp16, scaled by `by`, or (ROWS) each row at its own scale, which `scales` receives.
template <typename T, int DK, bool ROWS = false>
__device__ __forceinline__ void plane_halves(char* to, const char* from, float by, int thread, int threads, float* scales = nullptr) {
  using L = Lay<T, DK>;
  for (int i = 16 * thread; i < L::kRows; i += 16 * threads) {
    uint32_t x[L::kIn][4], y[L::kHalves][4];
#pragma unroll
    for (int n = 0; n < L::kIn; ++n) {
      const uint4 q = *reinterpret_cast<const uint4*>(from + n * L::kRows + i);
      x[n][0] = q.x; x[n][1] = q.y; x[n][2] = q.z; x[n][3] = q.w;
    }
    if (ROWS) {   // the largest of the first terms is within half a step of the row's; DK / 8 lanes have a row
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) most = max(most, max(x[0][e] << 16 & 0x7FFF0000u, x[0][e] & 0x7FFF0000u));
#pragma unroll
      for (int o = 1; o < DK / 8; o <<= 1) most = max(most, __shfl_xor_sync(~0u, most, o));
      const Scale row = plane_scale(most);
      by = row.to;
      scales[i / (2 * DK)] = row.from;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t t[L::kHalves];
      to_halves<L::kIn, L::kHalves>(x, e, by, t);
#pragma unroll
      for (int n = 0; n < L::kHalves; ++n) y[n][e] = t[n];
    }
#pragma unroll
    for (int n = 0; n < L::kHalves; ++n) *reinterpret_cast<uint4*>(to + n * L::kRows + i) = make_uint4(y[n][0], y[n][1], y[n][2], y[n][3]);
  }
}

// Decays between the tokens of a chunk: D_ij = e^{b_i - b_j} = row_i col_j for j in front of i's block of 16, with
// row_i = e^{b_i - m}, col_j = e^{m - b_j}, m the sum in front of the block; neither exceeds 1.
template <int C>
struct Decays {
  float row[C], col[C / 16][C];
  float key[C], value[C];   // beta e^b, beta: weights of T's columns
};

// A pair of T's columns c, c + 1 in row r.
template <int PITCH>
__device__ __forceinline__ float2 pair_at(const float* m, int r, int c) {
  return *reinterpret_cast<const float2*>(m + r * PITCH + c);
}

// Blocks T_ij = -T_ii sum_{j <= m < i} L_im T_mj (j < i) from the inverses T_ii of the diagonal blocks, one warp a
// block column j.  It works on the transposes, Z_i = -(sum Z_m L_im^T) T_ii^T, whose accumulators are the next product's A operand
// as they are; float32 in three terms.
template <int TILES, int PITCH>
__device__ __forceinline__ void invert_column(const float* L, float (&Z)[TILES][2][4], int j, int lane) {
  const int g = lane >> 2, t = 2 * (lane & 3);
  uint32_t za[TILES][3][4];
  auto turned = [&](int i, uint32_t (&b)[3][1][4], const float* at) {   // at [n][k] as a B operand
    const float2 x[4] = {pair_at<PITCH>(at, g, t), pair_at<PITCH>(at, g, t + 8), pair_at<PITCH>(at, g + 8, t), pair_at<PITCH>(at, g + 8, t + 8)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t s[3];
      split<3>(x[e].x, x[e].y, s);
#pragma unroll
      for (int n = 0; n < 3; ++n) b[n][0][e] = s[n];
    }
  };
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    if (i < j) continue;
    const float* diagonal = L + 16 * i * (PITCH + 1);
    if (i == j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = g + 8 * (e & 1), k = t + 8 * (e >> 1);
        uint32_t s[3];
        split<3>(diagonal[k * PITCH + r], diagonal[(k + 1) * PITCH + r], s);
#pragma unroll
        for (int n = 0; n < 3; ++n) za[i][n][e] = s[n];
      }
      continue;
    }
    Accumulators<2, true> acc;
    acc.clear();
    uint32_t b[3][1][4];
#pragma unroll
    for (int m = 0; m < TILES; ++m) {
      if (m < j || m >= i) continue;
      turned(i, b, L + 16 * i * PITCH + 16 * m);
      mma_terms(acc, 0, za[m], b);
    }
    float x[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = -acc.get(n, e);
    uint32_t xa[3][4];
    as_rows<3>(xa, x[0], x[1]);
    turned(i, b, diagonal);
    acc.clear();
    mma_terms(acc, 0, xa, b);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) Z[i][n][e] = acc.get(n, e);
    as_rows<3>(za[i], Z[i][0], Z[i][1]);
  }
}

// One chunk of one (b, h).  Half of the warps have what reads T from the left (K K^T, K^), the others the rest.
template <typename T, int DK, bool GRAD>
__global__ void __launch_bounds__(Prepare<T, DK>::kThreads, DK < 128 ? 3 : 1) delta_prepare(const __grid_constant__ Common p) {
  using P = Prepare<T, DK>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, TILES = L::kTiles, SIDES = L::kSides, THREADS = P::kThreads, PITCH = P::kPitch;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) typename L::M m;
  __shared__ __align__(16) Decays<C> w;
  __shared__ int32_t bad_key, bad;
  __shared__ uint32_t most, most_q, most_t;   // |k|, and for the gradients |q|, |T|
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t chunk = blockIdx.x % p.chunks;
  const int64_t bh = blockIdx.x / p.chunks, b = bh / p.H, h = bh % p.H, times = p.H / p.Hk, hk = h / times;
  const int64_t at = bh * p.chunks + chunk, at_key = (b * p.Hk + hk) * p.chunks + chunk;
  const int64_t t0 = static_cast<int64_t>(chunk) * C;
  const int rows = static_cast<int>(min(static_cast<int64_t>(C), p.N - t0));
  auto from = [&](const Operand& o, int64_t head) { return static_cast<const T*>(o.data) + b * o.sb + head * o.sh + t0 * o.sn; };
  float* inv = reinterpret_cast<float*>(smem);
  const uint32_t base = ptx::smem_u32(smem);
  const int strip = warp % TILES, m0 = 16 * strip, row = m0 + (lane >> 2);
  const bool second = warp >= TILES;

  Rows<T, DK, THREADS> k_units, q_units, v_units;
  k_units.fetch(from(p.k, hk), p.k.sn, rows, p.d, p.wide & kWideK);
  q_units.fetch(from(p.q, hk), p.q.sn, rows, p.d, p.wide & kWideQ);
  v_units.fetch(from(p.v, h), p.v.sn, rows, p.d, p.wide & kWideV);
  for (int i = threadIdx.x; i < DK; i += THREADS) m.first[i] = C;
  if (threadIdx.x == 0) {
    bad_key = bad = C;
    most = most_q = most_t = 0;
  }
  __syncthreads();

  // gates, E tokens a lane
  constexpr int E = C / 32;
  float g[E], beta[E];
  if (warp == 0) {
    const T *pg = from(p.g, h), *pb = from(p.beta, h);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = E * lane + e;
      g[e] = t < rows ? to_f(pg[t * p.g.sn]) : 0.0f;
      beta[e] = t < rows ? to_f(pb[t * p.beta.sn]) : 0.0f;
      g[e] = g[e] < kLowestGate ? kLowestGate : g[e];   // NaN stays
      if (!finite(g[e]) || !finite(beta[e])) atomicMin(&bad, t);
    }
  }
  load_rows<T, DK, THREADS, 1>(smem + P::kK, k_units, from(p.k, hk), p.k.sn, rows, p.d, p.wide & kWideK, &bad_key, &most);
  load_rows<T, DK, THREADS, 0, GRAD>(smem + P::kQ, q_units, from(p.q, hk), p.q.sn, rows, p.d, p.wide & kWideQ, nullptr, &most_q);
  load_rows<T, DK, THREADS, 2>(smem + P::kV, v_units, from(p.v, h), p.v.sn, rows, p.d, p.wide & kWideV, m.first);
  __syncthreads();
  if (warp == 0) {
    const int stop = min(bad, bad_key);
    Sum run[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = E * lane + e;
      if (t >= stop) g[e] = beta[e] = 0.0f;   // what follows is NaN anyway
      run[e] = gate_sum(g[e]);
      if (e) run[e] = add(run[e - 1], run[e]);
    }
    Sum all = run[E - 1];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      Sum o;
      o.hi = __shfl_up_sync(~0u, all.hi, s);
      o.lo = __shfl_up_sync(~0u, all.lo, s);
      if (lane >= s) all = add(o, all);
    }
    Sum before;
    before.hi = __shfl_up_sync(~0u, all.hi, 1);
    before.lo = __shfl_up_sync(~0u, all.lo, 1);
    if (lane == 0) before.hi = before.lo = 0.0f;
    auto of_lane = [&](int l) {
      Sum r;
      r.hi = __shfl_sync(~0u, all.hi, l);
      r.lo = __shfl_sync(~0u, all.lo, l);
      return r;
    };
    const Sum end = of_lane(31), none = {0.0f, 0.0f};
    Sum edge[TILES];
    edge[0] = none;
#pragma unroll
    for (int r = 1; r < TILES; ++r) edge[r] = of_lane(16 * r / E - 1);
    const int block = E * lane / 16;
    Sum mine = none;
#pragma unroll
    for (int r = 1; r < TILES; ++r)
      if (block == r) mine = edge[r];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = E * lane + e;
      const Sum s = add(before, run[e]);
      m.hi[t] = s.hi;
      m.lo[t] = s.lo;
      const float in = exp2_of(s, none);
      m.inside[t] = in;
      m.after[t] = exp2_of(end, s);
      m.beta[t] = beta[e];
      w.row[t] = exp2_of(s, mine);
      w.key[t] = t < stop ? beta[e] * in : 0.0f;
      w.value[t] = beta[e];
#pragma unroll
      for (int r = 1; r < TILES; ++r)
        if (r > block) w.col[r][t] = exp2_of(edge[r], s);
    }
    if (lane == 0) {
      m.total = exp2_of(end, none);
      m.key = scale_of(__uint_as_float(most)).from;
    }
  }
  __syncthreads();

  // K K^T (first) and Q K^T (second), 16 rows each, up to the diagonal
  {
    const uint32_t a_base = base + (second ? P::kQ : P::kK), b_base = base + P::kK;
    Accumulators<2 * TILES, L::kApart> acc;
    acc.clear();
#pragma unroll(L::kIn > 1 ? 1 : SIDES)
    for (int ks = 0; ks < SIDES; ++ks) {
      uint32_t a[L::kIn][4];
#pragma unroll
      for (int n = 0; n < L::kIn; ++n) a_rows<DK>(a[n], a_base + n * L::kRows, m0, 16 * ks, lane);
#pragma unroll
      for (int s = 0; s < TILES; ++s) {
        if (s > strip) continue;
        uint32_t x[L::kIn][1][4];
#pragma unroll
        for (int n = 0; n < L::kIn; ++n) b_rows<DK>(x[n][0], b_base + n * L::kRows, 16 * s, 16 * ks, lane);
        mma_terms(acc, 2 * s, a, x);
      }
    }
    if (second && !GRAD) {   // Q's rows, each at its own scale
      float most_q[2] = {0.0f, 0.0f};
      for (int ks = 0; ks < SIDES; ++ks) {
        uint32_t a[4];   // the first terms: the largest is within half a step of theirs
        a_rows<DK>(a, a_base, m0, 16 * ks, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) most_q[e & 1] = fmaxf(most_q[e & 1], fmaxf(fabsf(low(a[e])), fabsf(high(a[e]))));
      }
      const Scale by[2] = {scale_of(over_row(most_q[0])), scale_of(over_row(most_q[1]))};
      if ((lane & 3) == 0) {
        m.query[row] = p.scale * m.inside[row] * by[0].from;
        m.query[row + 8] = p.scale * m.inside[row + 8] * by[1].from;
      }
      if (h % times == 0)
        for (int ks = 0; ks < SIDES; ++ks) {
          uint32_t a[L::kIn][4], q[L::kHalves][4];
#pragma unroll
          for (int n = 0; n < L::kIn; ++n) a_rows<DK>(a[n], a_base + n * L::kRows, m0, 16 * ks, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t t[L::kHalves];
            to_halves<L::kIn, L::kHalves>(a, e, by[e & 1].to, t);
#pragma unroll
            for (int n = 0; n < L::kHalves; ++n) q[n][e] = t[n];
          }
#pragma unroll
          for (int n = 0; n < L::kHalves; ++n)
            *reinterpret_cast<uint4*>(p.im.q_rows + at_key * L::kInputHalf + ((strip * SIDES + ks) * L::kHalves + n) * kBlock + 16 * lane) =
                make_uint4(q[n][0], q[n][1], q[n][2], q[n][3]);
        }
    }
    const float f[2] = {w.row[row] * (second ? p.scale : m.beta[row]), w.row[row + 8] * (second ? p.scale : m.beta[row + 8])};
    float most_p[2] = {0.0f, 0.0f};
    float kept[GRAD ? 1 : TILES][2][4];   // the scores, until the largest of each row is known
#pragma unroll
    for (int s = 0; s < TILES; ++s) {
      float y[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int c = 16 * s + 8 * n + 2 * (lane & 3);
        if (s < strip) {
          const float2 x = *reinterpret_cast<const float2*>(w.col[strip] + c);
          y[n][0] = acc.get(2 * s + n, 0) * f[0] * x.x; y[n][1] = acc.get(2 * s + n, 1) * f[0] * x.y;
          y[n][2] = acc.get(2 * s + n, 2) * f[1] * x.x; y[n][3] = acc.get(2 * s + n, 3) * f[1] * x.y;
        } else if (s == strip) {
          const float2 h2 = *reinterpret_cast<const float2*>(m.hi + c), l2 = *reinterpret_cast<const float2*>(m.lo + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = row + 8 * (e >> 1), j = c + (e & 1);
            const Sum mine = {m.hi[r], m.lo[r]}, other = {e & 1 ? h2.y : h2.x, e & 1 ? l2.y : l2.x};
            const bool sees = second ? j <= r : j < r;
            y[n][e] = sees ? acc.get(2 * s + n, e) * exp2_of(mine, other) * (second ? p.scale : m.beta[r]) : 0.0f;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) y[n][e] = 0.0f;
        }
      }
      if (!second) {
        bool fine = true;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int c = 16 * s + 8 * n + 2 * (lane & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e) fine &= finite(y[n][e]);
          *reinterpret_cast<float2*>(inv + row * PITCH + c) = make_float2(y[n][0], y[n][1]);
          *reinterpret_cast<float2*>(inv + (row + 8) * PITCH + c) = make_float2(y[n][2], y[n][3]);
        }
        if (!fine)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!finite(y[n][e])) atomicMin(&bad, row + 8 * (e >> 1));
      } else if (GRAD && s <= strip) {
        uint32_t a[kChain][4];
        as_rows<kChain>(a, y[0], y[1]);
#pragma unroll
        for (int n = 0; n < kChain; ++n)   // columns in front of rows
          *reinterpret_cast<uint4*>(p.im.scores_back + at * L::kScoresBack + ((s * TILES + strip) * kChain + n) * kBlock + 16 * lane) =
              make_uint4(turn(a[n][0]), turn(a[n][1]), turn(a[n][2]), turn(a[n][3]));
      } else if (!GRAD) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            kept[GRAD ? 0 : s][n][e] = y[n][e];
            most_p[e >> 1] = fmaxf(most_p[e >> 1], fabsf(y[n][e]));
          }
      }
    }
    if (second && !GRAD) {
      const Scale by[2] = {scale_of(over_row(most_p[0])), scale_of(over_row(most_p[1]))};
      if ((lane & 3) == 0) {
        m.score[row] = by[0].from;
        m.score[row + 8] = by[1].from;
      }
#pragma unroll
      for (int s = 0; s < TILES; ++s) {
        if (s > strip) continue;
        uint32_t a[L::kHalves][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float(&y)[4] = kept[GRAD ? 0 : s][e >> 1];
          uint32_t t[L::kHalves];
          halves<L::kHalves>(y[2 * (e & 1)] * by[e & 1].to, y[2 * (e & 1) + 1] * by[e & 1].to, t);
#pragma unroll
          for (int n = 0; n < L::kHalves; ++n) a[n][e] = t[n];
        }
#pragma unroll
        for (int n = 0; n < L::kHalves; ++n)
          *reinterpret_cast<uint4*>(p.im.scores + at * L::kScores + ((strip * TILES + s) * L::kHalves + n) * kBlock + 16 * lane) =
              make_uint4(a[n][0], a[n][1], a[n][2], a[n][3]);
      }
    }
  }
  __syncthreads();
  const int stop = min(bad, bad_key);
  if (stop < C) {   // rows from there on write nothing
    for (int i = threadIdx.x; i < C * C; i += THREADS)
      if (i / C >= stop) inv[i / C * PITCH + i % C] = 0.0f;
    for (int i = threadIdx.x; i < C; i += THREADS)
      if (i >= stop) w.key[i] = w.value[i] = m.beta[i] = 0.0f;
    __syncthreads();
  }

  // T = (1 + L)^-1 in place: the diagonal blocks by columns, the others block by block
  if (!second && lane < 16) {
    float* block = inv + m0 * (PITCH + 1);
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) x[r] = r == lane ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 15; ++j)
#pragma unroll
      for (int r = j + 1; r < 16; ++r) x[r] = fmaf(-block[r * PITCH + j], x[j], x[r]);
    __syncwarp(0xFFFFu);
#pragma unroll
    for (int r = 0; r < 16; ++r) block[r * PITCH + lane] = x[r];
  }
  if (!second) ptx::named_bar_sync(1, THREADS / 2);   // the diagonal blocks are inverted; the other warps have the images meanwhile
  if (second && h % times == 0) {   // the key head's images, by its first head
    const float by = scale_of(__uint_as_float(most)).to;
    auto put = [&](char* to, const uint32_t (&x)[L::kIn][4]) {
      uint32_t k[L::kHalves][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t t[L::kHalves];
        to_halves<L::kIn, L::kHalves>(x, e, by, t);
#pragma unroll
        for (int n = 0; n < L::kHalves; ++n) k[n][e] = t[n];
      }
#pragma unroll
      for (int n = 0; n < L::kHalves; ++n) *reinterpret_cast<uint4*>(to + n * kBlock + 16 * lane) = make_uint4(k[n][0], k[n][1], k[n][2], k[n][3]);
    };
#pragma unroll 2
    for (int i = strip; i < SIDES * TILES; i += TILES) {
      const int side = i / TILES, ks = i % TILES;
      uint32_t x[L::kIn][4];
#pragma unroll
      for (int n = 0; n < L::kIn; ++n) b_cols<DK>(x[n], base + P::kK + n * L::kRows, 16 * side, 16 * ks, lane);
      put(p.im.k_add + at_key * L::kInputHalf + i * L::kHalves * kBlock, x);
      if (GRAD) {
#pragma unroll
        for (int n = 0; n < L::kIn; ++n) b_rows<DK>(x[n], base + P::kK + n * L::kRows, 16 * ks, 16 * side, lane);
        put(p.im.k_rows + at_key * L::kInputHalf + (ks * SIDES + side) * L::kHalves * kBlock, x);
#pragma unroll
        for (int n = 0; n < L::kIn; ++n) {
          b_cols<DK>(x[n], base + P::kQ + n * L::kRows, 16 * side, 16 * ks, lane);
          *reinterpret_cast<uint4*>(p.im.q_add + at_key * L::kInput + (i * L::kIn + n) * kBlock + 16 * lane) =
              make_uint4(x[n][0], x[n][1], x[n][2], x[n][3]);
        }
      }
    }
    if (GRAD) {
      plane_halves<T, DK>(p.im.k + at_key * L::kInputHalf, smem + P::kK, by, threadIdx.x - THREADS / 2, THREADS / 2);
      plane_halves<T, DK>(p.im.q + at_key * L::kInputHalf, smem + P::kQ, plane_scale(most_q).to, threadIdx.x - THREADS / 2, THREADS / 2);
    }
  }
  {
    float Z[TILES][2][4];
    if (!second) invert_column<TILES, PITCH>(inv, Z, strip, lane);
    __syncthreads();   // every warp has read L
    if (!second)
#pragma unroll
      for (int i = 1; i < TILES; ++i)
        if (i > strip)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) inv[(16 * i + 8 * n + 2 * (lane & 3) + (e & 1)) * PITCH + row + 8 * (e >> 1)] = Z[i][n][e];
  }
  __syncthreads();

  // T's rows of this strip with weighed columns: the A operand of K^ (first), the B operand of U^T (second)
  uint32_t a[TILES][kChain][4];
#pragma unroll
  for (int ks = 0; ks < TILES; ++ks) {
    if (ks > strip) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = row + 8 * (second ? e >> 1 : e & 1), c = 16 * ks + 2 * (lane & 3) + 8 * (second ? e & 1 : e >> 1);
      const float2 x = pair_at<PITCH>(inv, r, c), f = *reinterpret_cast<const float2*>((second ? w.value : w.key) + c);
      uint32_t t[kChain];
      split<kChain>(x.x * f.x, x.y * f.y, t);
#pragma unroll
      for (int n = 0; n < kChain; ++n) a[ks][n][e] = t[n];
    }
  }
  auto weighed = [&](Accumulators<2, true>& acc, int side) {
    acc.clear();
#pragma unroll
    for (int ks = 0; ks < TILES; ++ks) {
      if (ks > strip) continue;
      uint32_t x[L::kIn][4];
#pragma unroll
      for (int n = 0; n < L::kIn; ++n) {
        if (second)
          a_cols<DK>(x[n], base + P::kV + n * L::kRows, 16 * side, 16 * ks, lane);
        else
          b_cols<DK>(x[n], base + P::kK + n * L::kRows, 16 * side, 16 * ks, lane);
      }
      if (second) {
        uint32_t y[kChain][1][4];
#pragma unroll
        for (int n = 0; n < kChain; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[n][0][e] = a[ks][n][e];
        mma_terms(acc, 0, x, y);
      } else {
        uint32_t y[L::kIn][1][4];
#pragma unroll
        for (int n = 0; n < L::kIn; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[n][0][e] = x[n][e];
        mma_terms(acc, 0, a[ks], y);
      }
    }
  };
  if (second) {
#pragma unroll 1
    for (int side = 0; side < SIDES; ++side) {
      Accumulators<2, true> acc;
      weighed(acc, side);
      float4* to = reinterpret_cast<float4*>(p.im.u + (at * SIDES + side) * L::kTokens + 2 * strip * kBlock) + lane;
#pragma unroll
      for (int n = 0; n < 2; ++n) to[32 * n] = make_float4(acc.get(n, 0), acc.get(n, 1), acc.get(n, 2), acc.get(n, 3));
    }
  } else {   // kept in U's place until the largest of the strip is known: this warp's own bytes
    float largest = 0.0f;
    float4* keep = reinterpret_cast<float4*>(smem + P::kKeep) + (strip * SIDES * 64) + lane;
#pragma unroll 1
    for (int side = 0; side < SIDES; ++side) {
      Accumulators<2, true> acc;
      weighed(acc, side);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float4 y = make_float4(acc.get(n, 0), acc.get(n, 1), acc.get(n, 2), acc.get(n, 3));
        largest = fmaxf(largest, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
        keep[64 * side + 32 * n] = y;
      }
    }
    const Scale by = scale_of(__uint_as_float(__reduce_max_sync(~0u, __float_as_uint(largest))));
    if (lane == 0) m.keys[strip] = by.from;
#pragma unroll 1
    for (int side = 0; side < SIDES; ++side) {
      uint32_t k[2][4];   // rows of 16 tokens as A would have them; B takes the middle two the other way round
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float4 y = keep[64 * side + 32 * n];
        uint32_t t[2];
        halves<2>(y.x * by.to, y.y * by.to, t);
        k[0][2 * n] = t[0]; k[1][2 * n] = t[1];
        halves<2>(y.z * by.to, y.w * by.to, t);
        k[0][2 * n + 1] = t[0]; k[1][2 * n + 1] = t[1];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        *reinterpret_cast<uint4*>(p.im.keys + at * L::kKeys + ((strip * SIDES + side) * 2 + n) * kBlock + 16 * lane) =
            make_uint4(k[n][0], k[n][2], k[n][1], k[n][3]);
        if (GRAD)
          *reinterpret_cast<uint4*>(p.im.keys_add + at * L::kKeys + ((side * TILES + strip) * 2 + n) * kBlock + 16 * lane) =
              make_uint4(turn(k[n][0]), turn(k[n][1]), turn(k[n][2]), turn(k[n][3]));
      }
    }
  }
  if (GRAD) {   // T, and the rows of dout in V's place
    Rows<T, DK, THREADS> units;
    units.fetch(from(p.dout, h), p.dout.sn, rows, p.d, p.wide & kWideDout);
    float largest = 0.0f;
    auto each = [&](auto use) {
      for (int i = threadIdx.x; i < C * C / 2; i += THREADS) {
        const int r = i / (C / 2), c = 2 * (i % (C / 2));
        if (c <= (r | 15)) use(r, c, pair_at<PITCH>(inv, r, c));
      }
    };
    each([&](int, int, float2 x) { largest = fmaxf(largest, fmaxf(fabsf(x.x), fabsf(x.y))); });
    largest = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(largest)));
    if (lane == 0) atomicMax(&most_t, __float_as_uint(largest));
    __syncthreads();
    load_rows<T, DK, THREADS, 0>(smem + P::kV, units, from(p.dout, h), p.dout.sn, rows, p.d, p.wide & kWideDout, nullptr);
    const Scale by = plane_scale(most_t);
    each([&](int r, int c, float2 x) {
      uint32_t t[L::kHalves];
      halves<L::kHalves>(x.x * by.to, x.y * by.to, t);
#pragma unroll
      for (int n = 0; n < L::kHalves; ++n)
        *reinterpret_cast<uint32_t*>(p.im.inverse + at * L::kInverse + n * L::kSquare + unit_at<C>(r, c >> 3) + (c & 7) * 2) = t[n];
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      m.inverse = by.from;
      m.queries = plane_scale(most_q).from;
    }
    plane_halves<T, DK, true>(p.im.dout + at * L::kInputHalf, smem + P::kV, 0.0f, threadIdx.x, THREADS, m.douts);
    for (int i = warp; i < SIDES * TILES; i += 2 * TILES)
#pragma unroll
      for (int n = 0; n < L::kIn; ++n) {
        uint32_t x[4];
        a_cols<DK>(x, base + P::kV + n * L::kRows, 16 * (i / TILES), 16 * (i % TILES), lane);
        *reinterpret_cast<uint4*>(p.im.dout_cols + at * L::kInput + (i * L::kIn + n) * kBlock + 16 * lane) =
            make_uint4(x[0], x[1], x[2], x[3]);
      }
  }
  // marks
  bool any = false;
  for (int i = threadIdx.x; i < DK; i += THREADS) {
    m.first[i] = min(m.first[i], stop);
    any |= m.first[i] < C;
  }
  any = __syncthreads_or(any);
  if (threadIdx.x == 0) m.any = any;
  __syncthreads();
  for (int i = 16 * threadIdx.x; i < L::kMarks; i += 16 * THREADS)
    *reinterpret_cast<uint4*>(p.im.marks + at * L::kMarks + i) = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(&m) + i);
}

// A CTA walks the chunks with 16 MT columns of the state.  TILES warps make the chain: each forms the W of 16 tokens, and then its
// share of the state's rows.  The warps beside them fetch what all read, chunks ahead, and form 16 tokens' outputs, so nothing else
// stands between the chain's products: it waits for two barriers a chunk.  KEEP leaves the states and the w of every chunk for the
// gradients instead of outputs, with one warp beside each of the chain's.
template <typename T, int DK, int MT, bool KEEP>
struct ScanLay {
  using L = Lay<T, DK>;
  using M = typename L::M;
  static constexpr int kWarps = L::kTiles, kThreads = (KEEP ? 64 : 96) * kWarps;   // the chain's; with those beside it
  static constexpr int kShare = DK / 16 < kWarps ? 1 : DK / 16 / kWarps;   // blocks of the state's rows a warp
  static constexpr int kStatePlane = 16 * MT * DK * 2, kTokenPlane = 16 * MT * L::C * 2;
  // the state, e^{B-b} W and (for the outputs) W, and the scales of their rows
  static constexpr int kState = 0, kAfter = kState + 2 * kStatePlane, kW = kAfter + 2 * kTokenPlane;
  static constexpr int kStateScale = kW + (KEEP ? 0 : L::kHalves * kTokenPlane), kAfterScale = kStateScale + 16 * MT * L::kSides * 4;
  static constexpr int kTokenScales = 16 * MT * L::kTiles * 4, kWScale = kAfterScale + kTokenScales;
  static constexpr int kRing = (kWScale + (KEEP ? 0 : kTokenScales) + 127) / 128 * 128;
  // of a chunk, a pair of warps': blocks of K^, U, K, and of Q and the scores
  static constexpr int kKeysBytes = L::kSides * 2 * kBlock, kUBytes = 2 * kBlock, kAddBytes = kShare * L::kTiles * L::kHalves * kBlock;
  static constexpr int kQBytes = KEEP ? 0 : L::kSides * L::kHalves * kBlock, kScoreBytes = KEEP ? 0 : L::kTiles * L::kHalves * kBlock;
  static constexpr int kU = kKeysBytes, kAdd = kU + MT * kUBytes, kQ = kAdd + kAddBytes, kScores = kQ + kQBytes, kPair = kScores + kScoreBytes;
  static constexpr int kMarkFrom = offsetof(M, query), kMarkBytes = offsetof(M, first) - kMarkFrom;
  static constexpr int kMarks = kWarps * kPair, kStage = kMarks + (kMarkBytes + 127) / 128 * 128;
  static constexpr int kStages = (227 * 1024 - 1024 - kRing) / kStage < 3 ? 2 : 3;
  static constexpr int kBytes = kRing + kStages * kStage;
  static_assert(kBytes <= 226 * 1024, "shared memory");
  static_assert(kMarkFrom % 16 == 0 && kMarkBytes % 16 == 0 && kPair % 128 == 0, "copied in units of 16 bytes");
};

template <typename T, int DK, int MT, bool KEEP>
__global__ void __launch_bounds__(ScanLay<T, DK, MT, KEEP>::kThreads) delta_scan(const __grid_constant__ ScanArgs a) {
  using W = ScanLay<T, DK, MT, KEEP>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, TILES = L::kTiles, SIDES = L::kSides, SHARE = W::kShare, STAGES = W::kStages;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t bars[TILES][STAGES];
  const Common& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.d + 16 * MT - 1) / (16 * MT);
  const int64_t bh = blockIdx.x / groups, b = bh / p.H, h = bh % p.H, key = b * p.Hk + h / (p.H / p.Hk);
  const int tile0 = static_cast<int>(blockIdx.x % groups) * MT;
  const uint32_t base = ptx::smem_u32(smem), state = base + W::kState;
  const int count = static_cast<int>(p.chunks);
  const int own = warp % TILES;
  const int g = lane >> 2, t = 2 * (lane & 3);
  const bool shares = own * SHARE < SIDES;   // a warp of the chain has rows of the state
  auto sync = [&]() { ptx::named_bar_sync(1, W::kThreads); };   // of the CTA, from several places in the code
  // a chunk's marks from `query` on
  auto marks_at = [&](const char* stage) { return reinterpret_cast<const typename L::M*>(stage + W::kMarks - W::kMarkFrom); };
  // each column's first token that is not finite, where there is one
  auto first_of = [&](int i) { return reinterpret_cast<const typename L::M*>(p.im.marks + (bh * p.chunks + i) * L::kMarks)->first; };

  if (warp >= TILES) {
    const int part = warp / TILES - 1;   // half of the outputs' columns; the first also fetches
    uint64_t* bar = bars[own];
    if (part == 0 && lane == 0) {
#pragma unroll
      for (int n = 0; n < STAGES; ++n) ptx::mbar_init(bar + n, 1);
      ptx::fence_mbar_init();
    }
    __syncwarp();
    int alive = count;   // chunks; -1 - i once the wait for chunk i has given up
    const char* keys = p.im.keys + bh * p.chunks * L::kKeys + own * W::kKeysBytes;
    const char* u = p.im.u + (bh * p.chunks * SIDES + tile0) * L::kTokens + own * W::kUBytes;
    const char* add = p.im.k_add + key * p.chunks * L::kInputHalf + own * W::kAddBytes;
    const char* q_rows = KEEP ? nullptr : p.im.q_rows + key * p.chunks * L::kInputHalf + own * W::kQBytes;
    const char* scores = KEEP ? nullptr : p.im.scores + bh * p.chunks * L::kScores + own * W::kScoreBytes;
    const char* marks = p.im.marks + bh * p.chunks * L::kMarks + W::kMarkFrom;
    const uint32_t seen = KEEP ? 0 : (own + 1) * L::kHalves * kBlock;   // scores up to the diagonal
    const uint32_t bytes = W::kKeysBytes + MT * W::kUBytes + (shares ? W::kAddBytes : 0) + W::kQBytes + seen + (own == 0 ? W::kMarkBytes : 0);
    auto load = [&](int i) {
      if (part != 0 || lane != 0 || i >= alive) return;
      char* stage = smem + W::kRing + i % STAGES * W::kStage;
      char* to = stage + own * W::kPair;
      uint64_t* on = bar + i % STAGES;
      ptx::mbar_arrive_expect_tx(on, bytes);
      ptx::bulk_load_plain(to, keys, W::kKeysBytes, on);
#pragma unroll
      for (int n = 0; n < MT; ++n) ptx::bulk_load_plain(to + W::kU + n * W::kUBytes, u + n * L::kTokens, W::kUBytes, on);
      if (shares) ptx::bulk_load_plain(to + W::kAdd, add, W::kAddBytes, on);
      if (!KEEP) {
        ptx::bulk_load_plain(to + W::kQ, q_rows, W::kQBytes, on);
        ptx::bulk_load_plain(to + W::kScores, scores, seen, on);
        q_rows += L::kInputHalf;
        scores += L::kScores;
      }
      if (own == 0) ptx::bulk_load_plain(stage + W::kMarks, marks, W::kMarkBytes, on);
      keys += L::kKeys;
      u += SIDES * L::kTokens;
      add += L::kInputHalf;
      marks += L::kMarks;
    };
    for (int i = 0; i < STAGES - 1; ++i) load(i);
    if (part == 0 && stall_this_warp()) wait_copies_long(bar, 0, &g_delta_error);   // a test's
    T* const out = static_cast<T*>(a.out.data) + b * a.out.sb + h * a.out.sh;
    for (int i = 0; i < count; ++i) {
      const char* stage = smem + W::kRing + i % STAGES * W::kStage;
      const char* st = stage + own * W::kPair;
      if (part == 0 && alive >= 0 && !wait_copies(bar + i % STAGES, i / STAGES & 1, &g_delta_error)) alive = -1 - i;
      sync();   // the chunk's operands and the state's planes are there; the chunk before is done with
      load(i + STAGES - 1);
      if constexpr (KEEP) {
        sync();
      } else {
        // O = scale e^b Q S + scores W, this warp's 16 tokens and 8 MT columns
        const int col0 = 8 * MT * part;
        const auto* m = marks_at(stage);
        const float2 of_q = make_float2(m->query[16 * own + g], m->query[16 * own + g + 8]);
        const float2 of_p = make_float2(m->score[16 * own + g], m->score[16 * own + g + 8]);
        const int any = m->any;
        // a step of 16 of k has its own scale in each column
        float o[MT][4] = {};
        auto add_step = [&](const uint32_t (&q)[L::kHalves][4], uint32_t plane, int bytes, const float* scales, int steps, int ks, bool rows_of_state) {
          uint32_t x[L::kHalves][4];
#pragma unroll
          for (int k = 0; k < L::kHalves; ++k) {
            if (rows_of_state)
              b_rows<DK>(x[k], plane + k * bytes, 16 * (MT - 1) * part, 16 * ks, lane);
            else
              b_rows<C>(x[k], plane + k * bytes, 16 * (MT - 1) * part, 16 * ks, lane);
            if (MT == 1 && part) {
              x[k][0] = x[k][2];
              x[k][1] = x[k][3];
            }
          }
#pragma unroll
          for (int f = 0; f < MT; ++f) {
            float c[4];
            products(c, q, x, f);
            const float s0 = scales[(col0 + 8 * f + t) * steps + ks], s1 = scales[(col0 + 8 * f + t + 1) * steps + ks];
            o[f][0] = fmaf(c[0], s0, o[f][0]); o[f][1] = fmaf(c[1], s1, o[f][1]);
            o[f][2] = fmaf(c[2], s0, o[f][2]); o[f][3] = fmaf(c[3], s1, o[f][3]);
          }
        };
        const float *state_scale = reinterpret_cast<const float*>(smem + W::kStateScale), *token_scale = reinterpret_cast<const float*>(smem + W::kWScale);
#pragma unroll
        for (int ks = 0; ks < SIDES; ++ks) {
          uint32_t q[L::kHalves][4];
#pragma unroll
          for (int k = 0; k < L::kHalves; ++k) load_block(q[k], st + W::kQ, ks * L::kHalves + k, lane);
          add_step(q, state, W::kStatePlane, state_scale, SIDES, ks, true);
        }
        float of_state[MT][4];
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            of_state[n][e] = o[n][e] * (e < 2 ? of_q.x : of_q.y);
            o[n][e] = 0.0f;
          }
        sync();   // W's planes are there, the state's are read
#pragma unroll
        for (int ks = 0; ks < TILES; ++ks) {
          if (ks > own) continue;
          uint32_t q[L::kHalves][4];
#pragma unroll
          for (int k = 0; k < L::kHalves; ++k) load_block(q[k], st + W::kScores, ks * L::kHalves + k, lane);
          add_step(q, base + W::kW, W::kTokenPlane, token_scale, TILES, ks, false);
        }
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] = fmaf(o[n][e], e < 2 ? of_p.x : of_p.y, of_state[n][e]);
        const int64_t t0 = static_cast<int64_t>(i) * C;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int r = 16 * own + g + 8 * f;
          if (t0 + r >= p.N) continue;
#pragma unroll
          for (int n = 0; n < MT; ++n) {
            const int c = 16 * tile0 + col0 + 8 * n + t;
            if (c >= p.d) continue;
            float y[2] = {o[n][2 * f], o[n][2 * f + 1]};
            if (any)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (r >= first_of(i)[c + e]) y[e] = nan_value();
            store_pair<T>(out + (t0 + r) * a.out.sn + c, y[0], y[1], a.out_pairs, c + 1 < p.d);
          }
        }
      }
    }
#pragma unroll 1
    for (int j = -1 - alive; part == 0 && alive < 0 && j < min(-alive - 2 + STAGES, count); ++j)
      wait_copies_long(bar + j % STAGES, j / STAGES & 1, &g_delta_error);
    return;
  }

  // S^T: rows the state's columns 16 (tile0 + n) + g, + 8; columns this warp's share of its rows
  float S[MT][2 * SHARE][4];
  auto publish = [&]() {   // as planes of fp16 pairs, 16 columns of a row at a scale
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < SHARE; ++j)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float x[4] = {S[n][2 * j][2 * f], S[n][2 * j][2 * f + 1], S[n][2 * j + 1][2 * f], S[n][2 * j + 1][2 * f + 1]};
          const Scale by = scale_of(over_row(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])))));
          const int row = 16 * n + g + 8 * f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t h[2];
            halves<2>(x[2 * e] * by.to, x[2 * e + 1] * by.to, h);
            char* to = smem + W::kState + unit_at<DK>(row, 2 * (own * SHARE + j) + e) + 2 * t;
            *reinterpret_cast<uint32_t*>(to) = h[0];
            *reinterpret_cast<uint32_t*>(to + W::kStatePlane) = h[1];
          }
          if ((lane & 3) == 0) reinterpret_cast<float*>(smem + W::kStateScale)[row * SIDES + own * SHARE + j] = by.from;
        }
  };
  if (shares) {
    const float* in = a.init ? a.init + bh * p.d * p.d : nullptr;
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * own * SHARE + 8 * j + t + (e & 1), c = 16 * (tile0 + n) + g + 8 * (e >> 1);
          S[n][j][e] = in && r < p.d && c < p.d ? in[static_cast<int64_t>(r) * p.d + c] : 0.0f;
        }
    publish();
  }
  for (int i = 0; i < count; ++i) {
    const char* stage = smem + W::kRing + i % STAGES * W::kStage;
    const char* st = stage + own * W::kPair;
    const auto* m = marks_at(stage);
    sync();   // the chunk's operands and the state's planes are there; W's planes of the chunk before are read
    float w[MT][2][4];
    {
      // W^T = U^T - S^T K^^T, this warp's 16 tokens; a step of 16 of k has its own scale in each row, and the next step's operands
      // are asked for in front of a step's products
      float acc[MT][2][4] = {};
      uint32_t x[2][2][1][2][4], s[2][2][MT][2][4];
      auto fetch = [&](int pair) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ks = 2 * pair + h;
#pragma unroll
          for (int k = 0; k < 2; ++k) load_block(x[pair & 1][h][0][k], st, ks * 2 + k, lane);
#pragma unroll
          for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) a_rows<DK>(s[pair & 1][h][n][k], state + k * W::kStatePlane, 16 * n, 16 * ks, lane);
        }
      };
      const float* scales = reinterpret_cast<const float*>(smem + W::kStateScale) + g * SIDES;
      fetch(0);
#pragma unroll
      for (int pair = 0; pair < SIDES / 2; ++pair) {
        if (pair + 1 < SIDES / 2) fetch(pair + 1);
        add_scaled<MT, 2, 2, 2>(acc, s[pair & 1], x[pair & 1], [&](int k, int n) {
          return make_float2(scales[16 * n * SIDES + 2 * pair + k], scales[(16 * n + 8) * SIDES + 2 * pair + k]);
        });
      }
      const float of_keys = m->keys[own];
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 u = *reinterpret_cast<const float4*>(st + W::kU + (2 * n + j) * kBlock + 16 * lane);
          w[n][j][0] = fmaf(-of_keys, acc[n][j][0], u.x); w[n][j][1] = fmaf(-of_keys, acc[n][j][1], u.y);
          w[n][j][2] = fmaf(-of_keys, acc[n][j][2], u.z); w[n][j][3] = fmaf(-of_keys, acc[n][j][3], u.w);
        }
    }
    const float2 after[2] = {*reinterpret_cast<const float2*>(m->after + 16 * own + t), *reinterpret_cast<const float2*>(m->after + 16 * own + 8 + t)};
    const float total = m->total;
    // e^{B-b} W, which reaches the state, and W each at its own scale: where a chunk fades towards its end the first is far below the
    // second, and at W's scale would end below fp16's last bit
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        float x[4], z[4], most = 0.0f, most_z = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = w[n][e >> 1][2 * f + (e & 1)];
          z[e] = x[e] * (e & 1 ? after[e >> 1].y : after[e >> 1].x);
          most = fmaxf(most, fabsf(x[e]));
          most_z = fmaxf(most_z, fabsf(z[e]));
        }
        const Scale by_z = scale_of(over_row(most_z)), by = KEEP ? by_z : scale_of(over_row(most));
        const int row = 16 * n + g + 8 * f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int to = unit_at<C>(row, 2 * own + j) + 2 * t;
          uint32_t h[2];
          halves<2>(z[2 * j] * by_z.to, z[2 * j + 1] * by_z.to, h);
#pragma unroll
          for (int k = 0; k < 2; ++k) *reinterpret_cast<uint32_t*>(smem + W::kAfter + k * W::kTokenPlane + to) = h[k];
          if (!KEEP) {
            uint32_t y[L::kHalves];
            halves<L::kHalves>(x[2 * j] * by.to, x[2 * j + 1] * by.to, y);
#pragma unroll
            for (int k = 0; k < L::kHalves; ++k) *reinterpret_cast<uint32_t*>(smem + W::kW + k * W::kTokenPlane + to) = y[k];
          }
        }
        if ((lane & 3) == 0) {
          reinterpret_cast<float*>(smem + W::kAfterScale)[row * TILES + own] = by_z.from;
          if (!KEEP) reinterpret_cast<float*>(smem + W::kWScale)[row * TILES + own] = by.from;
        }
      }
    sync();   // W's planes are there, the state's are read
    if (KEEP)
#pragma unroll
      for (int n = 0; n < MT; ++n)
        if (16 * (tile0 + n) < p.d) {
          float4* to = reinterpret_cast<float4*>(p.im.w + ((bh * p.chunks + i) * SIDES + tile0 + n) * L::kTokens + 2 * own * kBlock) + lane;
#pragma unroll
          for (int j = 0; j < 2; ++j) to[32 * j] = make_float4(w[n][j][0], w[n][j][1], w[n][j][2], w[n][j][3]);
        }
    if (!shares) continue;
    // S^T <- e^B S^T + (e^{B-b} W)^T K, added outside the tensor core, which truncates what it adds
    float sum[MT][2 * SHARE][4] = {};
    {
      uint32_t x[2][2][SHARE][L::kHalves][4], v[2][2][MT][2][4];
      auto fetch = [&](int pair) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ks = 2 * pair + h;
#pragma unroll
          for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) a_rows<C>(v[pair & 1][h][n][k], base + W::kAfter + k * W::kTokenPlane, 16 * n, 16 * ks, lane);
#pragma unroll
          for (int j = 0; j < SHARE; ++j)
#pragma unroll
            for (int k = 0; k < L::kHalves; ++k) load_block(x[pair & 1][h][j][k], st + W::kAdd, (j * TILES + ks) * L::kHalves + k, lane);
        }
      };
      const float* scales = reinterpret_cast<const float*>(smem + W::kAfterScale) + g * TILES;
      fetch(0);
#pragma unroll
      for (int pair = 0; pair < TILES / 2; ++pair) {
        if (pair + 1 < TILES / 2) fetch(pair + 1);
        add_scaled<MT, 2 * SHARE, 2, L::kHalves>(sum, v[pair & 1], x[pair & 1], [&](int k, int n) {
          return make_float2(scales[16 * n * TILES + 2 * pair + k], scales[(16 * n + 8) * TILES + 2 * pair + k]);
        });
      }
    }
    const float of_key = m->key;
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j) {
        if (KEEP && 16 * (tile0 + n) < p.d)
          *reinterpret_cast<float4*>(p.im.s + ((bh * p.chunks + i) * SIDES + tile0 + n) * L::kState + (2 * own * SHARE + j) * kBlock + 16 * lane) =
              make_float4(S[n][j][0], S[n][j][1], S[n][j][2], S[n][j][3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[n][j][e] = fmaf(total, S[n][j][e], of_key * sum[n][j][e]);
      }
    if (m->any) {
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int c = 16 * (tile0 + n) + g + 8 * f;
          if (c < p.d && first_of(i)[c] < C)
#pragma unroll
            for (int j = 0; j < 2 * SHARE; ++j) S[n][j][2 * f] = S[n][j][2 * f + 1] = nan_value();
        }
    }
    publish();
  }
  if (shares && a.last) {
    float* last = a.last + bh * p.d * p.d;
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * own * SHARE + 8 * j + t + (e & 1), c = 16 * (tile0 + n) + g + 8 * (e >> 1);
          if (r < p.d && c < p.d) last[static_cast<int64_t>(r) * p.d + c] = S[n][j][e];
        }
  }
}

bool wide_rows(const Operand& o, int d, int dtype) {
  const int e = dtype == MHLA_BF16 ? 8 : 4;
  return d % e == 0 && reinterpret_cast<uintptr_t>(o.data) % 16 == 0 && o.sb % e == 0 && o.sn % e == 0 && o.sh % e == 0;
}

template <typename T, int DK, bool GRAD>
int prepare_as(const Common& c, int64_t BH, cudaStream_t s) {
  using P = Prepare<T, DK>;
  if (cudaFuncSetAttribute(delta_prepare<T, DK, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  KernelTimer timer("delta_prepare", s);
  delta_prepare<T, DK, GRAD><<<static_cast<unsigned>(BH * c.chunks), P::kThreads, P::kBytes, s>>>(c);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, int MT, bool KEEP>
int scan_as(const ScanArgs& a, int64_t BH, cudaStream_t s) {
  using W = ScanLay<T, DK, MT, KEEP>;
  static_assert(W::kBytes <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(delta_scan<T, DK, MT, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  const int groups = (a.c.d + 16 * MT - 1) / (16 * MT);
  KernelTimer timer(KEEP ? "delta_states" : "delta_scan", s);
  delta_scan<T, DK, MT, KEEP><<<static_cast<unsigned>(BH * groups), W::kThreads, W::kBytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK>
int scan_for(const ScanArgs& a, int64_t BH, bool keep, cudaStream_t s) {
  if constexpr (DK == 64 && sizeof(T) == 2)
    if (two_tiles(BH, a.c.d, kSms)) return keep ? scan_as<T, DK, 2, true>(a, BH, s) : scan_as<T, DK, 2, false>(a, BH, s);
  return keep ? scan_as<T, DK, 1, true>(a, BH, s) : scan_as<T, DK, 1, false>(a, BH, s);
}

template <typename T>
int prepare_type(const Common& c, int64_t BH, bool grad, cudaStream_t s) {
  switch (padded(c.d)) {
    case 32: return grad ? prepare_as<T, 32, true>(c, BH, s) : prepare_as<T, 32, false>(c, BH, s);
    case 64: return grad ? prepare_as<T, 64, true>(c, BH, s) : prepare_as<T, 64, false>(c, BH, s);
    default: return grad ? prepare_as<T, 128, true>(c, BH, s) : prepare_as<T, 128, false>(c, BH, s);
  }
}

template <typename T>
int scan_type(const ScanArgs& a, int64_t BH, bool keep, cudaStream_t s) {
  switch (padded(a.c.d)) {
    case 32: return scan_for<T, 32>(a, BH, keep, s);
    case 64: return scan_for<T, 64>(a, BH, keep, s);
    default: return scan_for<T, 128>(a, BH, keep, s);
  }
}

template <typename T, int DK>
size_t lay_out_as(int64_t heads, int64_t keys, bool grad, char* base, Images* im) {
  using L = Lay<T, DK>;
  size_t used = 0;
  auto take = [&](int64_t bytes) {
    char* at = base + used;
    used += align_up(static_cast<size_t>(bytes));
    return at;
  };
  im->k_add = take(keys * L::kInputHalf);
  im->keys = take(heads * L::kKeys);
  im->u = take(heads * L::kSides * L::kTokens);
  im->marks = take(heads * L::kMarks);
  if (!grad) {
    im->q_rows = take(keys * L::kInputHalf);
    im->scores = take(heads * L::kScores);
    return used;
  }
  im->k = take(keys * L::kInputHalf);
  im->q = take(keys * L::kInputHalf);
  im->dout = take(heads * L::kInputHalf);
  im->inverse = take(heads * L::kInverse);
  im->k_rows = take(keys * L::kInputHalf);
  im->keys_add = take(heads * L::kKeys);
  im->q_add = take(keys * L::kInput);
  im->scores_back = take(heads * L::kScoresBack);
  im->dout_cols = take(heads * L::kInput);
  im->s = take(heads * L::kSides * L::kState);
  im->ds = take(heads * L::kSides * L::kState);
  im->w = take(heads * L::kSides * L::kTokens);
  im->dw = take(heads * L::kSides * L::kTokens);
  return used;
}

template <typename T>
size_t lay_out_type(const DeltaProblem& p, int64_t chunks, bool grad, char* base, Images* im) {
  const int64_t heads = p.B * p.H * chunks, keys = p.B * p.Hk * chunks;
  switch (padded(p.d)) {
    case 32: return lay_out_as<T, 32>(heads, keys, grad, base, im);
    case 64: return lay_out_as<T, 64>(heads, keys, grad, base, im);
    default: return lay_out_as<T, 128>(heads, keys, grad, base, im);
  }
}

}  // namespace

int64_t delta_chunks(const DeltaProblem& p) {
  const int64_t C = p.dtype == MHLA_BF16 ? Form<__nv_bfloat16>::kChunk : Form<float>::kChunk;
  return (p.N + C - 1) / C;
}

namespace delta {

// Measured, bf16 at 4096 tokens (scan / gradients' chain, us, one tile against two): 192 tiles of d = 64 147 / 178 against 107 /
// 126, 384 of them 218 / 264 against 207 / 247, but 128 of them, which all run at once, 76 / 92 against 107 / 126; d = 32, where
// several CTAs of one tile fit on an SM, 384 of 2048 tokens 78 / 117 against 86 / 154 (when one warp stood beside each of the chain's).  float32
// at 2048 tokens, d = 64: 192 tiles 85 / 96 against 99 / 125, 384 of them 161 / 186 against 193 / 148.  So the scan takes two for bf16
// alone, and the gradients' chain beyond `most`, as many tiles as there are SMs for bf16 and twice as many for float32.  Heads of
// 65 to 128 channels take one: two were not measured.
bool two_tiles(int64_t BH, int d, int64_t most) { return d > 32 && BH * ((d + 15) / 16) > most; }

int launch_prepare(const Common& c, int64_t BH, int dtype, bool grad, cudaStream_t s) {
  return dtype == MHLA_BF16 ? prepare_type<__nv_bfloat16>(c, BH, grad, s) : prepare_type<float>(c, BH, grad, s);
}

int launch_scan(const ScanArgs& a, int64_t BH, int dtype, bool keep, cudaStream_t s) {
  return dtype == MHLA_BF16 ? scan_type<__nv_bfloat16>(a, BH, keep, s) : scan_type<float>(a, BH, keep, s);
}

size_t lay_out(const DeltaProblem& p, bool grad, char* base, Images* im) {
  return p.dtype == MHLA_BF16 ? lay_out_type<__nv_bfloat16>(p, delta_chunks(p), grad, base, im)
                              : lay_out_type<float>(p, delta_chunks(p), grad, base, im);
}

bool pairs_fit(const Operand& o, int d, int dtype) {
  const uintptr_t e = dtype == MHLA_BF16 ? 4 : 8;
  return d % 2 == 0 && reinterpret_cast<uintptr_t>(o.data) % e == 0 && o.sb % 2 == 0 && o.sn % 2 == 0 && o.sh % 2 == 0;
}

Common common(const DeltaProblem& p, const Operand* dout) {
  Common c = {};
  c.q = p.q; c.k = p.k; c.v = p.v; c.g = p.g; c.beta = p.beta;
  c.N = p.N; c.H = p.H; c.Hk = p.Hk;
  c.chunks = static_cast<uint32_t>(delta_chunks(p));
  c.d = p.d;
  c.scale = p.scale;
  c.wide = (wide_rows(p.q, p.d, p.dtype) ? kWideQ : 0) | (wide_rows(p.k, p.d, p.dtype) ? kWideK : 0) |
           (wide_rows(p.v, p.d, p.dtype) ? kWideV : 0);
  if (dout) {
    c.dout = *dout;
    if (wide_rows(*dout, p.d, p.dtype)) c.wide |= kWideDout;
  }
  return c;
}

}  // namespace delta

size_t delta_workspace_bytes(const DeltaProblem& p) {
  Images im;
  return lay_out(p, false, nullptr, &im);
}

int launch_delta_forward(const DeltaProblem& p, const float* state_in, const Operand& out, float* state_out, void* workspace,
                         void* stream) {
  ScanArgs a = {};
  a.c = common(p, nullptr);
  lay_out(p, false, static_cast<char*>(workspace), &a.c.im);
  a.init = state_in;
  a.last = state_out;
  a.out = out;
  a.out_pairs = pairs_fit(out, p.d, p.dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int rc = launch_prepare(a.c, p.B * p.H, p.dtype, false, s);
  return rc == MHLA_OK ? launch_scan(a, p.B * p.H, p.dtype, false, s) : rc;
}

// ------------------------------------------------------------------ one token

// The state is read and written once and nothing else is of size, so HBM bounds it.  A CTA takes SLICE columns of one (b, h):
// with y = S^T k and z = S^T q of the old state, w = beta (v - e^g y) and o = scale (e^g z + (q . k) w), so one pass over
// the rows gives both and the state stays in registers until it is written.
template <typename T, int VEC>
__global__ void __launch_bounds__(128) delta_step(const DeltaProblem p, float* state, const Operand out) {
  constexpr int SLICE = 8 * VEC, GROUPS = 16, MOST = 128 / GROUPS;   // columns, rows at once, rows a thread
  __shared__ float sq[128], sk[128];
  __shared__ float part[4][2][SLICE], dots[4];
  const int d = p.d, slices = (d + SLICE - 1) / SLICE;
  const int64_t bh = blockIdx.x / slices, b = bh / p.H, h = bh % p.H, hk = h / (p.H / p.Hk);
  const int x = threadIdx.x & 7, y = threadIdx.x >> 3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = static_cast<int>(blockIdx.x % slices) * SLICE + x * VEC;
  float* S = state + bh * d * d + c0;
  float s[MOST][VEC];
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int r = y + GROUPS * i;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[i][e] = 0.0f;
    if (r < d && c0 < d) {
      if constexpr (VEC == 4) {
        const float4 f = *reinterpret_cast<const float4*>(S + r * d);
        s[i][0] = f.x; s[i][1] = f.y; s[i][2] = f.z; s[i][3] = f.w;
      } else {
        s[i][0] = S[r * d];
      }
    }
  }
  auto at = [&](const Operand& o, int64_t head) { return static_cast<T*>(o.data) + b * o.sb + head * o.sh; };
  const int t = threadIdx.x;
  const float qt = t < d ? to_f(at(p.q, hk)[t]) : 0.0f, kt = t < d ? to_f(at(p.k, hk)[t]) : 0.0f;
  const float g = to_f(*at(p.g, h)), beta = to_f(*at(p.beta, h));
  const float decay = expf(g < kLowestGate ? kLowestGate : g);
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = c0 + e < d ? to_f(at(p.v, h)[c0 + e]) : 0.0f;
  sq[t] = qt;
  sk[t] = kt;
  float dot = qt * kt;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(~0u, dot, o);
  if (lane == 0) dots[warp] = dot;
  __syncthreads();
  float ky[VEC] = {}, qz[VEC] = {};
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int r = y + GROUPS * i;
    if (r >= d) break;
    const float k = sk[r], q = sq[r];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      ky[e] = fmaf(k, s[i][e], ky[e]);
      qz[e] = fmaf(q, s[i][e], qz[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    ky[e] += __shfl_xor_sync(~0u, ky[e], 8);
    ky[e] += __shfl_xor_sync(~0u, ky[e], 16);
    qz[e] += __shfl_xor_sync(~0u, qz[e], 8);
    qz[e] += __shfl_xor_sync(~0u, qz[e], 16);
    if (lane < 8) {
      part[warp][0][x * VEC + e] = ky[e];
      part[warp][1][x * VEC + e] = qz[e];
    }
  }
  __syncthreads();
  const float qk = (dots[0] + dots[1]) + (dots[2] + dots[3]);
  float w[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const int c = x * VEC + e;
    const float sum = (part[0][0][c] + part[1][0][c]) + (part[2][0][c] + part[3][0][c]);
    w[e] = beta * (v[e] - decay * sum);
    if (y == 0 && c0 + e < d) {
      const float z = (part[0][1][c] + part[1][1][c]) + (part[2][1][c] + part[3][1][c]);
      from_f(at(out, h) + c0 + e, p.scale * fmaf(decay, z, qk * w[e]));
    }
  }
#pragma unroll
  for (int i = 0; i < MOST; ++i) {
    const int r = y + GROUPS * i;
    if (r >= d || c0 >= d) break;
    const float k = sk[r];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[i][e] = fmaf(k, w[e], decay * s[i][e]);
    if constexpr (VEC == 4)
      *reinterpret_cast<float4*>(S + r * d) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    else
      S[r * d] = s[i][0];
  }
}

template <typename T, int VEC>
int step_as(const DeltaProblem& p, float* state, const Operand& out, cudaStream_t s) {
  const int slices = (p.d + 8 * VEC - 1) / (8 * VEC);
  KernelTimer timer("delta_step", s);
  delta_step<T, VEC><<<static_cast<unsigned>(p.B * p.H * slices), 128, 0, s>>>(p, state, out);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int launch_delta_step(const DeltaProblem& p, float* state, const Operand& out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = p.d % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
  if (p.dtype == MHLA_BF16) return vec ? step_as<__nv_bfloat16, 4>(p, state, out, s) : step_as<__nv_bfloat16, 1>(p, state, out, s);
  return vec ? step_as<float, 4>(p, state, out, s) : step_as<float, 1>(p, state, out, s);
}

int read_and_clear_delta_error(void* stream, uint32_t* flags) { return tc::read_and_clear_word(g_delta_error, stream, flags); }

MHLA_DEFINE_STALL_SETTER(set_stall_delta)

}  // namespace mhla
