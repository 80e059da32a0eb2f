// Root-mean-square norm of every query and key head with the position rotation
// in the same pass, and its gradients:
//   u = x / sqrt(mean(x^2) + eps),  y = u * weight,  z = R(position) y
//   dy = R^T dz,  dx = r (weight dy - u mean(u weight dy)),  dweight = sum dy u
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mhla_internal.h"

namespace mhla {
namespace {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
  for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// The rotation's row of a token, or -1 (unrotated), or -2 (past the table).
__device__ __forceinline__ int64_t rotation_row(const QkNormProblem& p, int64_t token) {
  if (!p.table) return -1;
  if (!p.positions) return token % p.N;
  const int64_t at = p.positions[token];
  return at < 0 ? -1 : at < p.rows ? at : -2;
}

struct Turn {
  float c, s;    // own channel: y c + partner s (the sign of the partner's term in s)
  int partner;
};

// Channel ch of a head: its pair's cos, signed sin and partner channel.
__device__ __forceinline__ Turn turn_of(const QkNormProblem& p, int64_t row, int ch) {
  if (row == -1 || ch >= 2 * p.pairs) return Turn{1.0f, 0.0f, ch};
  const int pair = p.interleaved ? ch >> 1 : (ch < p.pairs ? ch : ch - p.pairs);
  const bool second = p.interleaved ? ch & 1 : ch >= p.pairs;
  const int partner = p.interleaved ? ch ^ 1 : (second ? ch - p.pairs : ch + p.pairs);
  if (row == -2) return Turn{__int_as_float(0x7FC00000), 0.0f, partner};
  const float2 cs = reinterpret_cast<const float2*>(p.table)[row * p.pairs + pair];
  return Turn{cs.x, second ? cs.y : -cs.y, partner};
}

// One warp per head row; lane l holds channels l, l + 32, l + 64, l + 96.
template <typename T, bool BWD>
__global__ void __launch_bounds__(256) qk_norm_rows(const QkNormProblem p, float* part) {
  __shared__ float head[8][128];
  __shared__ float sums[BWD ? 2 * 128 * 8 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = p.Hq + p.Hk, rows = p.B * p.N * per;
  float* mine = head[warp];
  float acc[2][4] = {};
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + warp; i < rows; i += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t token = i / per, hh = i % per, b = token / p.N, n = token % p.N;
    const bool is_k = hh >= p.Hq;
    const int64_t h = is_k ? hh - p.Hq : hh;
    auto at = [&](const Operand& o) { return static_cast<T*>(o.data) + b * o.sb + n * o.sn + h * o.sh; };
    const T* x = at(is_k ? p.k : p.q);
    T* out = at(is_k ? p.k_out : p.q_out);
    const float* w = is_k ? p.k_weight : p.q_weight;
    const int64_t row = rotation_row(p, token);
    float v[4], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = lane + 32 * j;
      v[j] = ch < p.d ? to_f(x[ch]) : 0.0f;
      ss = fmaf(v[j], v[j], ss);
    }
    const float r = rsqrtf(warp_total(ss) / static_cast<float>(p.d) + p.eps);
    const T* dz = BWD ? at(is_k ? p.dk_out : p.dq_out) : nullptr;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = lane + 32 * j;
      v[j] *= r;
      if (ch < p.d) mine[ch] = BWD ? to_f(dz[ch]) : v[j] * (w ? w[ch] : 1.0f);
    }
    __syncwarp();
    float y[4], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = lane + 32 * j;
      y[j] = 0.0f;
      if (ch >= p.d) continue;
      const Turn t = turn_of(p, row, ch);
      y[j] = mine[ch] * t.c + mine[t.partner] * (BWD ? -t.s : t.s);
      if (BWD) {
        acc[is_k][j] += y[j] * v[j];
        y[j] *= w ? w[ch] : 1.0f;
        m = fmaf(y[j], v[j], m);
      }
    }
    if (BWD) m = warp_total(m) / static_cast<float>(p.d);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ch = lane + 32 * j;
      if (ch < p.d) from_f(out + ch, BWD ? r * (y[j] - v[j] * m) : y[j]);
    }
  }
  if (BWD) {
    for (int e = 0; e < 2; ++e)
      for (int j = 0; j < 4; ++j) sums[(e * 128 + lane + 32 * j) * 8 + warp] = acc[e][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 256; i += 256) {
      float s = 0.0f;
      for (int k = 0; k < 8; ++k) s += sums[i * 8 + k];
      part[static_cast<int64_t>(blockIdx.x) * 256 + i] = s;
    }
  }
}

// ------------------------------------------------------------------ eight channels a lane
//
// A head row is read once by a group of G lanes (G a power of two, the lanes behind
// the head's channels idle), each lane two runs of four channels chosen so that both
// channels of a pair are its own: no exchange for the rotation, and four pairs of the table a lane.
// A group takes kHeads heads of one token at a time, their loads in flight together and the
// rotation's row fetched once.  Every input byte is read once and every output byte written
// once: HBM bounds it.

// Four channels as loaded.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using Raw = float4;
  static __device__ __forceinline__ void expand(const Raw& r, float* x) {
    x[0] = r.x; x[1] = r.y; x[2] = r.z; x[3] = r.w;
  }
  static __device__ __forceinline__ Raw round(const float* x) { return make_float4(x[0], x[1], x[2], x[3]); }
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ void expand(const Raw& r, float* x) {
    x[0] = __uint_as_float(r.x << 16);
    x[1] = __uint_as_float(r.x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.y << 16);
    x[3] = __uint_as_float(r.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Raw round(const float* x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

template <int G>
__device__ __forceinline__ float group_total(float x) {
#pragma unroll
  for (int s = G / 2; s; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// (a, b) of every pair of a lane's channels x[0..3], x[4..7].
template <bool INTER>
__device__ __forceinline__ void turn(float (&x)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = INTER ? 2 * i : i, g = INTER ? 2 * i + 1 : i + 4;
    const float a = x[f], b = x[g];
    x[f] = fmaf(a, c[i], -s[i] * b);
    x[g] = fmaf(b, c[i], s[i] * a);
  }
}

struct Walk {
  int64_t items;            // (token, run of heads)
  int32_t runs_q, runs_k;   // runs of a token
  bool narrow;              // items and tokens in 32 bits
};

template <typename T, int G, bool BWD, bool INTER>
__global__ void __launch_bounds__(256, BWD ? 2 : 4) qk_norm_lanes(const QkNormProblem p, const Walk walk, float* part) {
  using R = typename Four<T>::Raw;
  constexpr int kHeads = BWD ? 3 : 4, kGroups = 256 / G;
  const int unit = threadIdx.x % G;
  const bool live = unit * 8 < p.d;
  // the lane's runs of channels; the four pairs 4 unit .. 4 unit + 3
  const bool pairs_here = !INTER && 4 * unit < p.pairs;
  const int c0 = pairs_here ? 4 * unit : 8 * unit, c1 = pairs_here ? 4 * unit + p.pairs : 8 * unit + 4;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const int runs = walk.runs_q + walk.runs_k;
  float acc[BWD ? 2 : 1][8] = {};
  // every lane of a warp takes the same number of rounds: the sums need all of them
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kGroups; i0 < walk.items; i0 += stride) {
    const int64_t i = i0 + threadIdx.x / G;
    const bool in = i < walk.items && live;
    const int64_t item = i < walk.items ? i : walk.items - 1;
    int64_t token, b;
    int run;
    if (walk.narrow) {
      const uint32_t t = static_cast<uint32_t>(item) / static_cast<uint32_t>(runs);
      run = static_cast<int>(static_cast<uint32_t>(item) - t * runs);
      b = t / static_cast<uint32_t>(p.N);
      token = t;
    } else {
      token = item / runs;
      run = static_cast<int>(item - token * runs);
      b = token / p.N;
    }
    const int64_t n = token - b * p.N;
    const bool is_k = run >= walk.runs_q;
    const int h0 = (is_k ? run - walk.runs_q : run) * kHeads;
    const int count = min(kHeads, static_cast<int>(is_k ? p.Hk : p.Hq) - h0);
    auto row_of = [&](const Operand& oq, const Operand& ok, int64_t& sh) {
      const Operand& o = is_k ? ok : oq;
      sh = o.sh;
      return static_cast<T*>(o.data) + b * o.sb + n * o.sn + h0 * o.sh;
    };
    int64_t xs, zs = 0, os;
    const T* x = row_of(p.q, p.k, xs);
    R xa[kHeads], xb[kHeads], za[BWD ? kHeads : 1], zb[BWD ? kHeads : 1];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      xa[j] = xb[j] = R{};
      if (in && j < count) {
        xa[j] = *reinterpret_cast<const R*>(x + j * xs + c0);
        xb[j] = *reinterpret_cast<const R*>(x + j * xs + c1);
      }
    }
    if (BWD) {
      const T* z = row_of(p.dq_out, p.dk_out, zs);
#pragma unroll
      for (int j = 0; j < kHeads; ++j) {
        za[BWD ? j : 0] = zb[BWD ? j : 0] = R{};
        if (in && j < count) {
          za[BWD ? j : 0] = *reinterpret_cast<const R*>(z + j * zs + c0);
          zb[BWD ? j : 0] = *reinterpret_cast<const R*>(z + j * zs + c1);
        }
      }
    }
    float c[4], s[4];
    const int64_t row = rotation_row(p, token);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = 1.0f;
      s[e] = 0.0f;
      if (row != -1 && 4 * unit + e < p.pairs) {
        const float2 cs = row == -2 ? make_float2(__int_as_float(0x7FC00000), 0.0f)
                                    : reinterpret_cast<const float2*>(p.table)[row * p.pairs + 4 * unit + e];
        c[e] = cs.x;
        s[e] = BWD ? -cs.y : cs.y;
      }
    }
    float w[8];
    const float* weight = is_k ? p.k_weight : p.q_weight;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = weight && live ? weight[(e < 4 ? c0 : c1) + (e & 3)] : 1.0f;
    T* out = row_of(p.q_out, p.k_out, os);
    float own[8] = {};   // the heads' share of the weight's gradient
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const bool real = in && j < count;
      float u[8], ss = 0.0f;
      Four<T>::expand(xa[j], u);
      Four<T>::expand(xb[j], u + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
      const float r = rsqrtf(group_total<G>(ss) * inv_d + p.eps);
      float y[8];
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = u[e] * r * w[e];
        turn<INTER>(y, c, s);
      } else {
        Four<T>::expand(za[BWD ? j : 0], y);
        Four<T>::expand(zb[BWD ? j : 0], y + 4);
        turn<INTER>(y, c, s);
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          u[e] *= r;
          if (real) own[e] = fmaf(y[e], u[e], own[e]);   // eps 0: a row that is not there is 0 / 0
          y[e] *= w[e];
          m = fmaf(y[e], u[e], m);
        }
        m = group_total<G>(m) * inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = r * (y[e] - u[e] * m);
      }
      if (real) {
        *reinterpret_cast<R*>(out + j * os + c0) = Four<T>::round(y);
        *reinterpret_cast<R*>(out + j * os + c1) = Four<T>::round(y + 4);
      }
    }
    if (BWD)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[0][e] += is_k ? 0.0f : own[e];
        acc[BWD ? 1 : 0][e] += is_k ? own[e] : 0.0f;
      }
  }
  if (BWD) {   // the block's sums, its groups in a fixed order
    __shared__ float sums[BWD ? kGroups * G * 8 : 1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
      float* mine = sums + (threadIdx.x / G) * G * 8;
      if (live)
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[(e < 4 ? c0 : c1) + (e & 3)] = acc[BWD ? k : 0][e];
      __syncthreads();
      if (threadIdx.x < p.d) {
        float t = 0.0f;
        for (int g = 0; g < kGroups; ++g) t += sums[g * G * 8 + threadIdx.x];
        part[static_cast<int64_t>(blockIdx.x) * 256 + k * 128 + threadIdx.x] = t;
      }
    }
  }
}

// Whether a lane's runs of four channels lie on the loads' boundaries and hold whole pairs.
bool in_lanes(const QkNormProblem& p, bool bwd) {
  if (p.d % 8 != 0 || (!p.interleaved && p.pairs % 4 != 0)) return false;
  const Operand* all[] = {&p.q, &p.k, &p.q_out, &p.k_out, &p.dq_out, &p.dk_out};
  const int64_t heads[] = {p.Hq, p.Hk, p.Hq, p.Hk, p.Hq, p.Hk};
  const uintptr_t bytes = p.dtype == MHLA_BF16 ? 8 : 16;
  for (int i = 0; i < (bwd ? 6 : 4); ++i) {
    if (heads[i] == 0) continue;
    const Operand& o = *all[i];
    if (reinterpret_cast<uintptr_t>(o.data) % bytes != 0 || o.sb % 4 != 0 || o.sn % 4 != 0 || o.sh % 4 != 0) return false;
  }
  return true;
}

constexpr int kBwdBlocks = 304;   // two CTAs an SM

template <typename T, int G, bool BWD>
unsigned launch_lanes_group(const QkNormProblem& p, float* part, cudaStream_t s) {
  constexpr int kHeads = BWD ? 3 : 4, kGroups = 256 / G;
  Walk w;
  w.runs_q = static_cast<int32_t>((p.Hq + kHeads - 1) / kHeads);
  w.runs_k = static_cast<int32_t>((p.Hk + kHeads - 1) / kHeads);
  w.items = p.B * p.N * (w.runs_q + w.runs_k);
  w.narrow = w.items < (int64_t{1} << 31) && p.N < (int64_t{1} << 31);
  const int64_t blocks = std::max<int64_t>(1, (w.items + kGroups - 1) / kGroups);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, BWD ? kBwdBlocks : int64_t{1} << 30));
  if (p.interleaved)
    qk_norm_lanes<T, G, BWD, true><<<grid, 256, 0, s>>>(p, w, part);
  else
    qk_norm_lanes<T, G, BWD, false><<<grid, 256, 0, s>>>(p, w, part);
  return grid;
}

template <bool BWD>
unsigned launch_lanes(const QkNormProblem& p, float* part, cudaStream_t s) {
  if (p.dtype == MHLA_BF16)
    return p.d <= 32   ? launch_lanes_group<__nv_bfloat16, 4, BWD>(p, part, s)
           : p.d <= 64 ? launch_lanes_group<__nv_bfloat16, 8, BWD>(p, part, s)
                       : launch_lanes_group<__nv_bfloat16, 16, BWD>(p, part, s);
  return p.d <= 32   ? launch_lanes_group<float, 4, BWD>(p, part, s)
         : p.d <= 64 ? launch_lanes_group<float, 8, BWD>(p, part, s)
                     : launch_lanes_group<float, 16, BWD>(p, part, s);
}

// One warp a channel: the blocks' sums in a fixed order.
__global__ void __launch_bounds__(256) qk_norm_weight_grad(const float* part, int blocks, int32_t d, float* dq_weight,
                                                           float* dk_weight) {
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int ch = i & 127;
  float* out = i < 128 ? dq_weight : dk_weight;
  if (ch >= d || !out) return;
  float s = 0.0f;
  for (int b = lane; b < blocks; b += 32) s += part[static_cast<int64_t>(b) * 256 + i];
  s = warp_total(s);
  if (lane == 0) out[ch] = s;
}

int64_t row_blocks(const QkNormProblem& p) {
  return std::max<int64_t>(1, (p.B * p.N * (p.Hq + p.Hk) + 7) / 8);
}

}  // namespace

size_t qk_norm_bwd_workspace_bytes(int32_t) { return align_up(static_cast<size_t>(kBwdBlocks) * 256 * 4); }

int launch_qk_norm(const QkNormProblem& p, void* stream) {
  KernelTimer timer("qk_norm", stream);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(row_blocks(p), 152 * 64));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (in_lanes(p, false))
    launch_lanes<false>(p, nullptr, s);
  else if (p.dtype == MHLA_BF16)
    qk_norm_rows<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p, nullptr);
  else
    qk_norm_rows<float, false><<<grid, 256, 0, s>>>(p, nullptr);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int launch_qk_norm_backward(const QkNormProblem& p, void* workspace, void* stream) {
  unsigned grid = static_cast<unsigned>(std::min<int64_t>(row_blocks(p), kBwdBlocks));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  {
    KernelTimer timer("qk_norm_backward", stream);
    const bool any = p.B > 0 && p.Hq + p.Hk > 0;   // the walk over lanes needs a row
    if (any && in_lanes(p, true))
      grid = launch_lanes<true>(p, part, s);
    else if (p.dtype == MHLA_BF16)
      qk_norm_rows<__nv_bfloat16, true><<<grid, 256, 0, s>>>(p, part);
    else
      qk_norm_rows<float, true><<<grid, 256, 0, s>>>(p, part);
    if (cudaGetLastError() != cudaSuccess) return MHLA_ERR_CUDA;
  }
  if (!p.dq_weight && !p.dk_weight) return MHLA_OK;
  KernelTimer timer("qk_norm_weight_grad", stream);
  qk_norm_weight_grad<<<32, 256, 0, s>>>(part, static_cast<int>(grid), p.d, p.dq_weight, p.dk_weight);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

}  // namespace mhla
