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
// The scan is a chain of two products a chunk, so latency bounds it.  It runs transposed: a warp holds 16
// columns of S as rows of S^T in its accumulators, and S^T K^^T, W^T and W^T K follow one another from accumulators to
// A operands without leaving its registers; no warp of the chain waits for another.  A second warp beside each forms the outputs
// of the chunk before from what the first left in shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "delta_common.cuh"

namespace mhla {

using namespace delta;

namespace {

// Rows of one operand to planes of terms; zeros behind the last token and channel.
// WATCH 1: the first row with a value that is not finite to `first`; 2: each column's; such values are left as zeros.
template <typename T, int DK, int THREADS, int WATCH>
__device__ __forceinline__ void load_rows(char* dst, const T* src, int64_t sn, int rows, int d, bool wide, int32_t* first) {
  using L = Lay<T, DK>;
  constexpr int C = L::C;
  auto watch = [&](float x, int r, int c) {
    if (WATCH == 0 || finite(x)) return x;
    atomicMin(first + (WATCH == 2 ? c : 0), r);
    return 0.0f;
  };
  if (wide) {
    constexpr int E = 16 / sizeof(T), kUnits = C * DK / E, kEach = kUnits / THREADS;
    static_assert(kUnits % THREADS == 0, "whole passes");
    uint4 x[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = threadIdx.x + THREADS * j, r = i / (DK / E), c = E * (i % (DK / E));
      x[j] = r < rows && c < d ? *reinterpret_cast<const uint4*>(src + r * sn + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int i = threadIdx.x + THREADS * j, r = i / (DK / E), c = E * (i % (DK / E));
      uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      if constexpr (sizeof(T) == 2) {
        if (WATCH != 0) {
          uint32_t bad = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {   // 0 times what is not finite is NaN
            const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), __floats2bfloat162_rn(0.0f, 0.0f));
            bad |= *reinterpret_cast<const uint32_t*>(&z);
          }
          if (bad & 0x7FFF7FFFu)
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
}

template <typename T, int DK, bool GRAD>
struct Prepare {
  using L = Lay<T, DK>;
  static constexpr int C = L::C, kStrips = C / 16, kThreads = 64 * kStrips;
  static constexpr int kPitch = C + 4, kHalf = C / 2 + 4;   // floats a row of T, of a product on the way
  static constexpr int kSum = 0, kTmp = kSum + C * kPitch * 4, kK = (kTmp + C / 2 * kHalf * 4 + 127) / 128 * 128;
  static constexpr int kV = kK + L::kInput, kQ = kV + L::kInput, kPlanes = kQ;   // T's planes where Q was
  static constexpr int kBytes = std::max(kQ + L::kInput, kPlanes + 2 * L::kInverse);
};

// T = (1 + L)^-1 of the strictly lower triangular L in place, float32: the diagonal blocks of 16 by columns, then
// blocks of twice the size, T21 = -T22 L21 T11.  All threads.
template <int C, int PITCH, int HALF, int THREADS>
__device__ __forceinline__ void invert(float* L, float* tmp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < C / 16 && lane < 16) {
    float* block = L + 16 * warp * (PITCH + 1);
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
  __syncthreads();
#pragma unroll
  for (int H = 16; H < C; H *= 2) {
    const int quads = H / 4, each = H * quads, n = C / (2 * H) * each;   // outputs in fours
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const int pair = i / each, r = i % each / quads, c = 4 * (i % quads);
      const float *a = L + (2 * H * pair + H + r) * PITCH + 2 * H * pair, *b = L + 2 * H * pair * (PITCH + 1) + c;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
      for (int k = 0; k < H; ++k) {
        const float x = a[k];
        const float4 y = *reinterpret_cast<const float4*>(b + k * PITCH);
        s.x = fmaf(x, y.x, s.x); s.y = fmaf(x, y.y, s.y); s.z = fmaf(x, y.z, s.z); s.w = fmaf(x, y.w, s.w);
      }
      *reinterpret_cast<float4*>(tmp + (H * pair + r) * HALF + c) = s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += THREADS) {
      const int pair = i / each, r = i % each / quads, c = 4 * (i % quads);
      const float *a = L + (2 * H * pair + H + r) * PITCH + 2 * H * pair + H, *b = tmp + H * pair * HALF + c;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
      for (int k = 0; k < H; ++k) {
        const float x = a[k];
        const float4 y = *reinterpret_cast<const float4*>(b + k * HALF);
        s.x = fmaf(-x, y.x, s.x); s.y = fmaf(-x, y.y, s.y); s.z = fmaf(-x, y.z, s.z); s.w = fmaf(-x, y.w, s.w);
      }
      *reinterpret_cast<float4*>(L + (2 * H * pair + H + r) * PITCH + 2 * H * pair + c) = s;
    }
    __syncthreads();
  }
}

// T with its columns weighed, as planes of terms, lower blocks of 16.
template <typename T, int DK, typename Weight>
__device__ __forceinline__ void put_inverse(char* dst, const float* inv, int pitch, int threads, Weight weight) {
  using L = Lay<T, DK>;
  constexpr int C = L::C;
  for (int i = threadIdx.x; i < C * C / 2; i += threads) {
    const int r = i / (C / 2), c = 2 * (i % (C / 2));
    if (c > (r | 15)) continue;
    const float2 x = *reinterpret_cast<const float2*>(inv + r * pitch + c);
    uint32_t t[L::kOwn];
    split<L::kOwn>(weight(x.x, c), weight(x.y, c + 1), t);
#pragma unroll
    for (int n = 0; n < L::kOwn; ++n)
      *reinterpret_cast<uint32_t*>(dst + n * L::kSquare + unit_at<C>(r, c >> 3) + (c & 7) * 2) = t[n];
  }
}

// One chunk of one (b, h).
template <typename T, int DK, bool GRAD>
__global__ void __launch_bounds__(Prepare<T, DK, GRAD>::kThreads) delta_prepare(const __grid_constant__ Common p) {
  using P = Prepare<T, DK, GRAD>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, THREADS = P::kThreads, PITCH = P::kPitch;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) typename L::M m;
  __shared__ int32_t bad_key, bad;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t chunk = blockIdx.x % p.chunks;
  const int64_t bh = blockIdx.x / p.chunks, b = bh / p.H, h = bh % p.H, times = p.H / p.Hk, hk = h / times;
  const int64_t at = bh * p.chunks + chunk, at_key = (b * p.Hk + hk) * p.chunks + chunk;
  const int64_t t0 = static_cast<int64_t>(chunk) * C;
  const int rows = static_cast<int>(min(static_cast<int64_t>(C), p.N - t0));
  auto from = [&](const Operand& o, int64_t head) { return static_cast<const T*>(o.data) + b * o.sb + head * o.sh + t0 * o.sn; };
  float* inv = reinterpret_cast<float*>(smem + P::kSum);
  const uint32_t base = ptx::smem_u32(smem);

  for (int i = threadIdx.x; i < DK; i += THREADS) m.first[i] = C;
  if (threadIdx.x == 0) bad_key = bad = C;
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
  load_rows<T, DK, THREADS, 1>(smem + P::kK, from(p.k, hk), p.k.sn, rows, p.d, p.wide & kWideK, &bad_key);
  load_rows<T, DK, THREADS, 0>(smem + P::kQ, from(p.q, hk), p.q.sn, rows, p.d, p.wide & kWideQ, nullptr);
  load_rows<T, DK, THREADS, 2>(smem + P::kV, from(p.v, h), p.v.sn, rows, p.d, p.wide & kWideV, m.first);
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
    Sum end;
    end.hi = __shfl_sync(~0u, all.hi, 31);
    end.lo = __shfl_sync(~0u, all.lo, 31);
    const Sum none = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = E * lane + e;
      const Sum s = add(before, run[e]);
      m.hi[t] = s.hi;
      m.lo[t] = s.lo;
      m.inside[t] = exp2_of(s, none);
      m.after[t] = exp2_of(end, s);
      m.beta[t] = beta[e];
    }
    if (lane == 0) m.total = exp2_of(end, none);
  }
  __syncthreads();

  // K K^T (first half of the warps) and Q K^T (second half), 16 rows each, up to the diagonal
  {
    const int strip = warp % P::kStrips, m0 = 16 * strip, row = m0 + (lane >> 2);
    const bool scores = warp >= P::kStrips;
    const uint32_t a_base = base + (scores ? P::kQ : P::kK), b_base = base + P::kK;
    Accumulators<2 * P::kStrips, L::kApart> acc;
    acc.clear();
#pragma unroll(L::kIn > 1 ? 1 : DK / 16)
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t a[L::kIn][4];
#pragma unroll
      for (int n = 0; n < L::kIn; ++n) a_rows<DK>(a[n], a_base + n * L::kRows, m0, 16 * ks, lane);
#pragma unroll
      for (int s = 0; s < P::kStrips; ++s) {
        if (s > strip) continue;
        uint32_t x[L::kIn][1][4];
#pragma unroll
        for (int n = 0; n < L::kIn; ++n) b_rows<DK>(x[n][0], b_base + n * L::kRows, 16 * s, 16 * ks, lane);
        mma_terms(acc, 2 * s, a, x);
      }
    }
    const Sum br[2] = {{m.hi[row], m.lo[row]}, {m.hi[row + 8], m.lo[row + 8]}};
    const float beta_r[2] = {m.beta[row], m.beta[row + 8]};
    char* img = p.im.scores + at * L::kScores;
#pragma unroll
    for (int n = 0; n < 2 * P::kStrips; ++n) {
      const int c = 8 * n + 2 * (lane & 3);
      float y[4] = {};
      if (n < 2 * strip + 2) {
        const float2 h2 = *reinterpret_cast<const float2*>(m.hi + c), l2 = *reinterpret_cast<const float2*>(m.lo + c);
        const Sum bc[2] = {{h2.x, l2.x}, {h2.y, l2.y}};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = row + 8 * (e >> 1), s = c + (e & 1);
          if (scores ? s <= r : s < r) {
            y[e] = acc.get(n, e) * exp2_of(br[e >> 1], bc[e & 1]) * (scores ? p.scale : beta_r[e >> 1]);
            if (!scores && !finite(y[e])) atomicMin(&bad, r);
          }
        }
      }
      if (scores) {
        if (n < 2 * strip + 2) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            uint32_t t[L::kScore];
            split<L::kScore>(y[2 * f], y[2 * f + 1], t);
#pragma unroll
            for (int k = 0; k < L::kScore; ++k)
              *reinterpret_cast<uint32_t*>(img + k * L::kSquare + unit_at<C>(row + 8 * f, n) + 4 * (lane & 3)) = t[k];
          }
        }
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f) *reinterpret_cast<float2*>(inv + (row + 8 * f) * PITCH + c) = make_float2(y[2 * f], y[2 * f + 1]);
      }
    }
  }
  __syncthreads();
  const int stop = min(bad, bad_key);
  if (stop < C) {   // rows from there on write nothing
    for (int i = threadIdx.x; i < C * C; i += THREADS)
      if (i / C >= stop) inv[i / C * PITCH + i % C] = 0.0f;
    for (int i = threadIdx.x; i < C; i += THREADS)
      if (i >= stop) m.beta[i] = 0.0f;
  }
  __syncthreads();

  // images of the rows, by the key head's first head
  if (h % times == 0) {
    for (int i = 16 * threadIdx.x; i < L::kInput; i += 16 * THREADS) {
      *reinterpret_cast<uint4*>(p.im.k + at_key * L::kInput + i) = *reinterpret_cast<const uint4*>(smem + P::kK + i);
      *reinterpret_cast<uint4*>(p.im.q + at_key * L::kInput + i) = *reinterpret_cast<const uint4*>(smem + P::kQ + i);
    }
  }
  invert<C, PITCH, P::kHalf, THREADS>(inv, reinterpret_cast<float*>(smem + P::kTmp));

  // the planes of T beta e^b and T beta take the place of Q, which every warp is through with
  char *with_decay = smem + P::kPlanes, *with_beta = with_decay + L::kInverse;
  put_inverse<T, DK>(with_decay, inv, PITCH, THREADS, [&](float x, int c) { return c < stop ? x * (m.beta[c] * m.inside[c]) : 0.0f; });
  put_inverse<T, DK>(with_beta, inv, PITCH, THREADS, [&](float x, int c) { return x * m.beta[c]; });
  if (GRAD) put_inverse<T, DK>(p.im.inverse + at * L::kInverse, inv, PITCH, THREADS, [&](float x, int) { return x; });
  __syncthreads();

  if (warp < P::kStrips) {   // K^ rows
    const int m0 = 16 * warp, row = m0 + (lane >> 2);
    char* img = p.im.keys + at * L::kKeys;
    constexpr int G = 2;   // pairs of column tiles at once
#pragma unroll 1
    for (int n0 = 0; n0 < DK; n0 += 16 * G) {
      Accumulators<2 * G, L::kApart> acc;
      acc.clear();
#pragma unroll
      for (int ks = 0; ks < P::kStrips; ++ks) {
        if (ks > warp) continue;
        uint32_t a[L::kOwn][4], x[L::kIn][G][4];
#pragma unroll
        for (int n = 0; n < L::kOwn; ++n) a_rows<C>(a[n], base + P::kPlanes + n * L::kSquare, m0, 16 * ks, lane);
#pragma unroll
        for (int n = 0; n < L::kIn; ++n)
#pragma unroll
          for (int j = 0; j < G; ++j) b_cols<DK>(x[n][j], base + P::kK + n * L::kRows, n0 + 16 * j, 16 * ks, lane);
        mma_terms(acc, 0, a, x);
      }
#pragma unroll
      for (int n = 0; n < 2 * G; ++n)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          uint32_t t[L::kOwn];
          split<L::kOwn>(acc.get(n, 2 * f), acc.get(n, 2 * f + 1), t);
#pragma unroll
          for (int k = 0; k < L::kOwn; ++k)
            *reinterpret_cast<uint32_t*>(img + k * L::kRows + unit_at<DK>(row + 8 * f, n0 / 8 + n) + 4 * (lane & 3)) = t[k];
        }
    }
  } else {                   // U^T, 16 columns of the values at a time
    const uint32_t with_beta_at = base + P::kPlanes + L::kInverse;
#pragma unroll 1
    for (int tile = warp - P::kStrips; tile < DK / 16; tile += P::kStrips) {
      if (16 * tile >= p.d) break;
      Accumulators<2 * P::kStrips, L::kApart> acc;
      acc.clear();
#pragma unroll
      for (int ks = 0; ks < P::kStrips; ++ks) {
        uint32_t a[L::kIn][4];
#pragma unroll
        for (int n = 0; n < L::kIn; ++n) a_cols<DK>(a[n], base + P::kV + n * L::kRows, 16 * tile, 16 * ks, lane);
#pragma unroll
        for (int s = ks; s < P::kStrips; ++s) {
          uint32_t x[L::kOwn][1][4];
#pragma unroll
          for (int n = 0; n < L::kOwn; ++n) b_rows<C>(x[n][0], with_beta_at + n * L::kSquare, 16 * s, 16 * ks, lane);
          mma_terms(acc, 2 * s, a, x);
        }
      }
      float4* to = reinterpret_cast<float4*>(p.im.u + (at * (DK / 16) + tile) * L::kTokens) + lane;
#pragma unroll
      for (int n = 0; n < 2 * P::kStrips; ++n) to[32 * n] = make_float4(acc.get(n, 0), acc.get(n, 1), acc.get(n, 2), acc.get(n, 3));
    }
  }
  if (GRAD) {   // rows of dout, in V's place
    __syncthreads();
    load_rows<T, DK, THREADS, 0>(smem + P::kV, from(p.dout, h), p.dout.sn, rows, p.d, p.wide & kWideDout, nullptr);
    __syncthreads();
    for (int i = 16 * threadIdx.x; i < L::kInput; i += 16 * THREADS)
      *reinterpret_cast<uint4*>(p.im.dout + at * L::kInput + i) = *reinterpret_cast<const uint4*>(smem + P::kV + i);
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

// NW warps of the chain (16 columns of the state each) and, unless KEEP, as many for the outputs.  KEEP leaves
// the states and the w of every chunk for the gradients instead.
template <typename T, int DK, int NW, bool KEEP>
struct ScanLay {
  using L = Lay<T, DK>;
  static constexpr int kThreads = (KEEP ? 32 : 64) * NW;
  static constexpr int kK = 0, kKeys = kK + L::kInput, kU = kKeys + L::kKeys, kMarks = kU + NW * L::kTokens;
  static constexpr int kStage = kMarks + L::kMarks;
  static constexpr int kQ = 0, kScores = kQ + L::kInput, kMarksOut = kScores + L::kScores, kStageOut = kMarksOut + L::kMarks;
  static constexpr int kHand = L::kState + L::kTokens;   // a warp's S and W of one chunk
  static constexpr int kOut = 2 * kStage, kHands = kOut + 2 * kStageOut;
  static constexpr int kBytes = KEEP ? 2 * kStage : kHands + 2 * NW * kHand;
};

template <typename T, int DK, int NW, bool KEEP>
__global__ void __launch_bounds__(ScanLay<T, DK, NW, KEEP>::kThreads) delta_scan(const __grid_constant__ ScanArgs a) {
  using W = ScanLay<T, DK, NW, KEEP>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, NT = C / 8, NS = DK / 8, THREADS = W::kThreads;
  extern __shared__ __align__(128) char smem[];
  const Common& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.d + 16 * NW - 1) / (16 * NW);
  const int64_t bh = blockIdx.x / groups, b = bh / p.H, h = bh % p.H, key = b * p.Hk + h / (p.H / p.Hk);
  const int tile0 = static_cast<int>(blockIdx.x % groups) * NW;
  const uint32_t base = ptx::smem_u32(smem);
  const int count = static_cast<int>(p.chunks);
  const int own = warp % NW, tile = tile0 + own, c0 = 16 * tile + (lane >> 2);
  const bool chain = KEEP || warp < NW;

  auto load = [&](int i) {
    const uint32_t st = base + (i & 1) * W::kStage;
    const int64_t at = bh * p.chunks + i;
    copy_async(st + W::kK, p.im.k + (key * p.chunks + i) * L::kInput, L::kInput, threadIdx.x, THREADS);
    copy_async(st + W::kKeys, p.im.keys + at * L::kKeys, L::kKeys, threadIdx.x, THREADS);
    copy_async(st + W::kU, p.im.u + (at * (DK / 16) + tile0) * L::kTokens, NW * L::kTokens, threadIdx.x, THREADS);
    copy_async(st + W::kMarks, p.im.marks + at * L::kMarks, L::kMarks, threadIdx.x, THREADS);
  };
  auto load_out = [&](int i) {
    const uint32_t st = base + W::kOut + (i & 1) * W::kStageOut;
    const int64_t at = bh * p.chunks + i;
    copy_async(st + W::kQ, p.im.q + (key * p.chunks + i) * L::kInput, L::kInput, threadIdx.x, THREADS);
    copy_async(st + W::kScores, p.im.scores + at * L::kScores, L::kScores, threadIdx.x, THREADS);
    copy_async(st + W::kMarksOut, p.im.marks + at * L::kMarks, L::kMarks, threadIdx.x, THREADS);
  };
  load(0);
  commit();

  // S^T: rows c0, c0 + 8 (columns of the state), columns 8 n + 2 (lane % 4) and the next
  float S[NS][4];
  if (chain) {
    const float* in = a.init ? a.init + bh * p.d * p.d : nullptr;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 8 * n + 2 * (lane & 3) + (e & 1), c = c0 + 8 * (e >> 1);
        S[n][e] = in && r < p.d && c < p.d ? in[static_cast<int64_t>(r) * p.d + c] : 0.0f;
      }
  }

  for (int i = 0; i < count + (KEEP ? 0 : 1); ++i) {
    wait_all();
    __syncthreads();
    if (i + 1 < count) load(i + 1);
    if (!KEEP && i < count) load_out(i);
    commit();
    if (chain) {
      if (i >= count) continue;
      const char* stage = smem + (i & 1) * W::kStage;
      const uint32_t st = base + (i & 1) * W::kStage;
      const auto& m = *reinterpret_cast<const typename L::M*>(stage + W::kMarks);
      // W^T = U^T - S^T K^^T
      Accumulators<NT, L::kApart> acc;
      acc.clear();
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t s[L::kOwn][4], x[L::kOwn][NT / 2][4];
        as_rows<L::kOwn>(s, S[2 * ks], S[2 * ks + 1]);
#pragma unroll
        for (int n = 0; n < L::kOwn; ++n)
#pragma unroll
          for (int j = 0; j < NT / 2; ++j) b_rows<DK>(x[n][j], st + W::kKeys + n * L::kRows, 16 * j, 16 * ks, lane);
        mma_terms(acc, 0, s, x);
      }
      float w[NT][4];
      {
        const float4* u = reinterpret_cast<const float4*>(stage + W::kU + own * L::kTokens) + lane;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float4 x = u[32 * n];
          w[n][0] = x.x - acc.get(n, 0); w[n][1] = x.y - acc.get(n, 1);
          w[n][2] = x.z - acc.get(n, 2); w[n][3] = x.w - acc.get(n, 3);
        }
      }
      {
        float4 *to_s, *to_w;
        if (KEEP) {
          const int64_t at = (bh * p.chunks + i) * (DK / 16) + tile;
          to_s = reinterpret_cast<float4*>(p.im.s + at * L::kState) + lane;
          to_w = reinterpret_cast<float4*>(p.im.w + at * L::kTokens) + lane;
        } else {
          char* hand = smem + W::kHands + ((i & 1) * NW + own) * W::kHand;
          to_s = reinterpret_cast<float4*>(hand) + lane;
          to_w = reinterpret_cast<float4*>(hand + L::kState) + lane;
        }
        if (!KEEP || 16 * tile < p.d) {
#pragma unroll
          for (int n = 0; n < NS; ++n) to_s[32 * n] = make_float4(S[n][0], S[n][1], S[n][2], S[n][3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) to_w[32 * n] = make_float4(w[n][0], w[n][1], w[n][2], w[n][3]);
        }
      }
      // S^T <- e^B S^T + (e^{B-b} W)^T K.  The chunk's sum is formed apart and added once, rounded to nearest: a long
      // sequence must not gather the tensor core's truncation.
      uint32_t wa[C / 16][L::kOwn][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 f = *reinterpret_cast<const float2*>(m.after + 8 * n + 2 * (lane & 3));
        w[n][0] *= f.x; w[n][1] *= f.y; w[n][2] *= f.x; w[n][3] *= f.y;
      }
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks) as_rows<L::kOwn>(wa[ks], w[2 * ks], w[2 * ks + 1]);
      const float total = m.total;
      constexpr int G = DK / 16 < 4 ? DK / 16 : 4;
#pragma unroll
      for (int n0 = 0; n0 < NS; n0 += 2 * G) {
        Accumulators<2 * G, L::kApart> sum;
        sum.clear();
#pragma unroll
        for (int ks = 0; ks < C / 16; ++ks) {
          uint32_t x[L::kIn][G][4];
#pragma unroll
          for (int n = 0; n < L::kIn; ++n)
#pragma unroll
            for (int j = 0; j < G; ++j) b_cols<DK>(x[n][j], st + W::kK + n * L::kRows, 8 * n0 + 16 * j, 16 * ks, lane);
          mma_terms(sum, 0, wa[ks], x);
        }
#pragma unroll
        for (int n = 0; n < 2 * G; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n0 + n][e] = fmaf(total, S[n0 + n][e], sum.get(n, e));
      }
      if (m.any) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          if (c0 + 8 * f < p.d && m.first[c0 + 8 * f] < C)
#pragma unroll
            for (int n = 0; n < NS; ++n) S[n][2 * f] = S[n][2 * f + 1] = nan_value();
      }
    } else if (!KEEP && i > 0) {
      // O = scale e^b Q S + scores W: rows of tokens, this warp's 16 columns
      const int done = i - 1;
      const char* stage = smem + W::kOut + (done & 1) * W::kStageOut;
      const uint32_t st = base + W::kOut + (done & 1) * W::kStageOut;
      const auto& m = *reinterpret_cast<const typename L::M*>(stage + W::kMarksOut);
      const char* hand = smem + W::kHands + ((done & 1) * NW + own) * W::kHand;
      const float4 *of_s = reinterpret_cast<const float4*>(hand) + lane,
                   *of_w = reinterpret_cast<const float4*>(hand + L::kState) + lane;
      Accumulators<2, L::kApart> o[C / 16];
#pragma unroll
      for (int s = 0; s < C / 16; ++s) o[s].clear();
#pragma unroll(L::kIn > 1 ? 1 : DK / 16)
      for (int ks = 0; ks < DK / 16; ++ks) {
        // a transposed accumulator is a B operand as it is: rows its columns, columns its k
        const float4 x = of_s[64 * ks], y = of_s[64 * ks + 32];
        uint32_t sb[L::kOwn][1][4], t[L::kOwn];
        auto put = [&](int e, float f, float g) {
          split<L::kOwn>(f, g, t);
#pragma unroll
          for (int n = 0; n < L::kOwn; ++n) sb[n][0][e] = t[n];
        };
        put(0, x.x, x.y); put(1, y.x, y.y); put(2, x.z, x.w); put(3, y.z, y.w);
#pragma unroll
        for (int s = 0; s < C / 16; ++s) {
          uint32_t q[L::kIn][4];
#pragma unroll
          for (int n = 0; n < L::kIn; ++n) a_rows<DK>(q[n], st + W::kQ + n * L::kRows, 16 * s, 16 * ks, lane);
          mma_terms(o[s], 0, q, sb);
        }
      }
#pragma unroll
      for (int s = 0; s < C / 16; ++s) {
        const float f0 = p.scale * m.inside[16 * s + (lane >> 2)], f1 = p.scale * m.inside[16 * s + (lane >> 2) + 8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[s].main[n][e] = o[s].get(n, e) * (e < 2 ? f0 : f1);
            if (L::kApart) o[s].small[L::kApart ? n : 0][e] = 0.0f;
          }
        }
      }
#pragma unroll
      for (int ks = 0; ks < C / 16; ++ks) {
        const float4 x = of_w[64 * ks], y = of_w[64 * ks + 32];
        uint32_t wb[L::kOwn][1][4], t[L::kOwn];
        auto put = [&](int e, float f, float g) {
          split<L::kOwn>(f, g, t);
#pragma unroll
          for (int n = 0; n < L::kOwn; ++n) wb[n][0][e] = t[n];
        };
        put(0, x.x, x.y); put(1, y.x, y.y); put(2, x.z, x.w); put(3, y.z, y.w);
#pragma unroll
        for (int s = ks; s < C / 16; ++s) {
          uint32_t q[L::kScore][4];
#pragma unroll
          for (int n = 0; n < L::kScore; ++n) a_rows<C>(q[n], st + W::kScores + n * L::kSquare, 16 * s, 16 * ks, lane);
          mma_terms(o[s], 0, q, wb);
        }
      }
      const int64_t t0 = static_cast<int64_t>(done) * C;
      T* out = static_cast<T*>(a.out.data) + b * a.out.sb + h * a.out.sh;
#pragma unroll
      for (int s = 0; s < C / 16; ++s)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int r = 16 * s + (lane >> 2) + 8 * f;
          if (t0 + r >= p.N) continue;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int c = 16 * tile + 8 * n + 2 * (lane & 3);
            if (c >= p.d) continue;
            float y[2] = {o[s].get(n, 2 * f), o[s].get(n, 2 * f + 1)};
            if (m.any)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (r >= m.first[c + e]) y[e] = nan_value();
            store_pair<T>(out + (t0 + r) * a.out.sn + c, y[0], y[1], a.out_pairs, c + 1 < p.d);
          }
        }
    }
  }
  if (chain && a.last) {
    float* last = a.last + bh * p.d * p.d;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 8 * n + 2 * (lane & 3) + (e & 1), c = c0 + 8 * (e >> 1);
        if (r < p.d && c < p.d) last[static_cast<int64_t>(r) * p.d + c] = S[n][e];
      }
  }
}

bool wide_rows(const Operand& o, int d, int dtype) {
  const int e = dtype == MHLA_BF16 ? 8 : 4;
  return d % e == 0 && reinterpret_cast<uintptr_t>(o.data) % 16 == 0 && o.sb % e == 0 && o.sn % e == 0 && o.sh % e == 0;
}

template <typename T, int DK, bool GRAD>
int prepare_as(const Common& c, int64_t BH, cudaStream_t s) {
  using P = Prepare<T, DK, GRAD>;
  if (cudaFuncSetAttribute(delta_prepare<T, DK, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  KernelTimer timer("delta_prepare", s);
  delta_prepare<T, DK, GRAD><<<static_cast<unsigned>(BH * c.chunks), P::kThreads, P::kBytes, s>>>(c);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, bool KEEP>
int scan_as(const ScanArgs& a, int64_t BH, cudaStream_t s) {
  constexpr int NW = 2;
  using W = ScanLay<T, DK, NW, KEEP>;
  static_assert(W::kBytes <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(delta_scan<T, DK, NW, KEEP>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  const int groups = (a.c.d + 16 * NW - 1) / (16 * NW);
  KernelTimer timer(KEEP ? "delta_states" : "delta_scan", s);
  delta_scan<T, DK, NW, KEEP><<<static_cast<unsigned>(BH * groups), W::kThreads, W::kBytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
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
    case 32: return keep ? scan_as<T, 32, true>(a, BH, s) : scan_as<T, 32, false>(a, BH, s);
    case 64: return keep ? scan_as<T, 64, true>(a, BH, s) : scan_as<T, 64, false>(a, BH, s);
    default: return keep ? scan_as<T, 128, true>(a, BH, s) : scan_as<T, 128, false>(a, BH, s);
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
  im->k = take(keys * L::kInput);
  im->q = take(keys * L::kInput);
  im->keys = take(heads * L::kKeys);
  im->scores = take(heads * L::kScores);
  im->u = take(heads * (DK / 16) * L::kTokens);
  im->marks = take(heads * L::kMarks);
  if (grad) {
    im->inverse = take(heads * L::kInverse);
    im->dout = take(heads * L::kInput);
    im->s = take(heads * (DK / 16) * L::kState);
    im->ds = take(heads * (DK / 16) * L::kState);
    im->w = take(heads * (DK / 16) * L::kTokens);
    im->dw = take(heads * (DK / 16) * L::kTokens);
  }
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

}  // namespace mhla
