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

// ------------------------------------------------------------------ 16-byte units
//
// A head row is read once, in 16-byte units, by a group of G lanes (G a power of two, the
// lanes behind the head's units idle), kHeads heads of a token at a time: the rotation's
// row is fetched once for them, and their loads are in flight together.  Every input
// byte is read once and every output byte written once, so HBM bounds it.

template <typename T>
struct Units;
template <>
struct Units<__nv_bfloat16> {
  static constexpr int kVec = 8;
};
template <>
struct Units<float> {
  static constexpr int kVec = 4;
};

__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 repack(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 repack(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

template <int G>
__device__ __forceinline__ float group_total(float x) {
#pragma unroll
  for (int s = G / 2; s; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// The turn of a lane's VEC channels: y[e] -> y[e] c[e] + partner s[e].
template <int VEC>
struct Turns {
  float c[VEC], s[VEC];
  int partner;        // lane that holds the partners (half layout)
};

template <int VEC, int G>
__device__ __forceinline__ Turns<VEC> turns_of(const QkNormProblem& p, int64_t row, int unit, int lane) {
  Turns<VEC> t;
  t.partner = lane;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    t.c[e] = 1.0f;
    t.s[e] = 0.0f;
  }
  if (!p.table) return t;
  const float2* cs = reinterpret_cast<const float2*>(p.table) + (row > 0 ? row * p.pairs : 0);
  const float nan = __int_as_float(0x7FC00000);
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const int pair = unit * (VEC / 2) + e / 2;
      if (pair >= p.pairs || row == -1) continue;
      const float2 x = row == -2 ? make_float2(nan, 0.0f) : cs[pair];
      t.c[e] = t.c[e + 1] = x.x;
      t.s[e] = -x.y;
      t.s[e + 1] = x.y;
    }
    return t;
  }
  const int half = p.pairs / VEC;   // units a half
  if (unit >= 2 * half) return t;
  const bool second = unit >= half;
  t.partner = second ? lane - half : lane + half;
  if (row == -1) return t;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const float2 x = row == -2 ? make_float2(nan, 0.0f) : cs[(second ? unit - half : unit) * VEC + e];
    t.c[e] = x.x;
    t.s[e] = second ? x.y : -x.y;
  }
  return t;
}

template <int VEC>
__device__ __forceinline__ void turn(float (&y)[VEC], const Turns<VEC>& t, bool interleaved, float sign) {
  float o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = interleaved ? y[e ^ 1] : __shfl_sync(~0u, y[e], t.partner);
#pragma unroll
  for (int e = 0; e < VEC; ++e) y[e] = fmaf(y[e], t.c[e], sign * t.s[e] * o[e]);
}

// kHeads heads of a token per group of G lanes; a grid-stride walk over (token, run of heads).
template <typename T, int G, bool BWD>
__global__ void __launch_bounds__(256) qk_norm_units(const QkNormProblem p, float* part) {
  constexpr int VEC = Units<T>::kVec, kHeads = BWD ? 2 : 4, kGroups = 256 / G;
  const int lane = threadIdx.x & 31, unit = threadIdx.x % G;
  const bool live = unit * VEC < p.d;
  const int64_t heads = p.Hq + p.Hk, runs = (heads + kHeads - 1) / kHeads, items = p.B * p.N * runs;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  float w[2][VEC], acc[2][VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    w[0][e] = p.q_weight && live ? p.q_weight[unit * VEC + e] : 1.0f;
    w[1][e] = p.k_weight && live ? p.k_weight[unit * VEC + e] : 1.0f;
    acc[0][e] = acc[1][e] = 0.0f;
  }
  // every lane of a warp takes the same number of rounds: the shuffles need all of them
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kGroups; i0 < items; i0 += stride) {
    const int64_t i = i0 + threadIdx.x / G;
    const bool in = i < items && live;
    const int64_t item = i < items ? i : items - 1;
    const int64_t token = item / runs, b = token / p.N, n = token - b * p.N;
    const int h0 = static_cast<int>(item - token * runs) * kHeads;
    uint4 x[kHeads], z[BWD ? kHeads : 1];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const bool is_k = h0 + j >= p.Hq;
      const int64_t h = is_k ? h0 + j - p.Hq : h0 + j;
      const bool has = in && h0 + j < heads;
      const Operand& src = is_k ? p.k : p.q;
      x[j] = has ? *reinterpret_cast<const uint4*>(static_cast<const T*>(src.data) + b * src.sb + n * src.sn +
                                                   h * src.sh + unit * VEC)
                 : zero;
      if (BWD) {
        const Operand& g = is_k ? p.dk_out : p.dq_out;
        z[j] = has ? *reinterpret_cast<const uint4*>(static_cast<const T*>(g.data) + b * g.sb + n * g.sn + h * g.sh +
                                                     unit * VEC)
                   : zero;
      }
    }
    const Turns<VEC> t = turns_of<VEC, G>(p, rotation_row(p, token), unit, lane);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const bool is_k = h0 + j >= p.Hq;
      const int64_t h = is_k ? h0 + j - p.Hq : h0 + j;
      const float(&ww)[VEC] = w[0];
      float u[VEC], ss = 0.0f;
      unpack(x[j], u);
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(u[e], u[e], ss);
      const float r = rsqrtf(group_total<G>(ss) * inv_d + p.eps);
      float y[VEC];
      if (!BWD) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = u[e] * r * (is_k ? w[1][e] : ww[e]);
        turn(y, t, p.interleaved, 1.0f);
      } else {
        unpack(z[BWD ? j : 0], y);
        turn(y, t, p.interleaved, -1.0f);
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          u[e] *= r;
          const float du = y[e] * u[e];
          if (is_k)
            acc[1][e] += du;
          else
            acc[0][e] += du;
          y[e] *= is_k ? w[1][e] : ww[e];
          m = fmaf(y[e], u[e], m);
        }
        m = group_total<G>(m) * inv_d;
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[e] = r * (y[e] - u[e] * m);
      }
      if (in && h0 + j < heads) {
        const Operand& dst = is_k ? p.k_out : p.q_out;
        *reinterpret_cast<uint4*>(static_cast<T*>(dst.data) + b * dst.sb + n * dst.sn + h * dst.sh + unit * VEC) =
            repack(y);
      }
    }
  }
  if (BWD) {   // the block's sums, its groups in a fixed order
    __shared__ float sums[BWD ? kGroups * G * VEC : 1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) sums[(threadIdx.x / G) * G * VEC + unit * VEC + e] = acc[k][e];
      __syncthreads();
      for (int c = threadIdx.x; c < 128; c += 256) {
        float s = 0.0f;
        if (c < G * VEC)
          for (int g = 0; g < kGroups; ++g) s += sums[g * G * VEC + c];
        part[static_cast<int64_t>(blockIdx.x) * 256 + k * 128 + c] = s;
      }
    }
  }
}

// Whether the call's rows and their pairs fall into whole 16-byte units.
bool in_units(const QkNormProblem& p, bool bwd) {
  const int vec = p.dtype == MHLA_BF16 ? 8 : 4;
  if (p.d % vec != 0 || (!p.interleaved && p.pairs % vec != 0)) return false;
  const Operand* all[] = {&p.q, &p.k, &p.q_out, &p.k_out, &p.dq_out, &p.dk_out};
  const int64_t heads[] = {p.Hq, p.Hk, p.Hq, p.Hk, p.Hq, p.Hk};
  for (int i = 0; i < (bwd ? 6 : 4); ++i) {
    if (heads[i] == 0) continue;
    const Operand& o = *all[i];
    if (reinterpret_cast<uintptr_t>(o.data) % 16 != 0 || o.sb % vec != 0 || o.sn % vec != 0 || o.sh % vec != 0)
      return false;
  }
  return p.Hq + p.Hk < (int64_t{1} << 30);
}

constexpr int kBwdBlocks = 608;   // four CTAs an SM

template <typename T, int G>
void launch_units_group(const QkNormProblem& p, bool bwd, float* part, unsigned* grid, cudaStream_t s) {
  const int64_t heads = p.Hq + p.Hk, per = bwd ? 2 : 4, groups = 256 / G;
  const int64_t items = p.B * p.N * ((heads + per - 1) / per);
  const int64_t blocks = std::max<int64_t>(1, (items + groups - 1) / groups);
  if (bwd) {
    *grid = static_cast<unsigned>(std::min<int64_t>(blocks, kBwdBlocks));
    qk_norm_units<T, G, true><<<*grid, 256, 0, s>>>(p, part);
  } else {
    *grid = static_cast<unsigned>(std::min<int64_t>(blocks, int64_t{1} << 30));
    qk_norm_units<T, G, false><<<*grid, 256, 0, s>>>(p, nullptr);
  }
}

template <typename T>
void launch_units(const QkNormProblem& p, bool bwd, float* part, unsigned* grid, cudaStream_t s) {
  const int units = p.d / Units<T>::kVec;
  if (units <= 4)
    launch_units_group<T, 4>(p, bwd, part, grid, s);
  else if (units <= 8)
    launch_units_group<T, 8>(p, bwd, part, grid, s);
  else if (units <= 16)
    launch_units_group<T, 16>(p, bwd, part, grid, s);
  else if constexpr (sizeof(T) == 4)
    launch_units_group<T, 32>(p, bwd, part, grid, s);
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
  unsigned grid = static_cast<unsigned>(std::min<int64_t>(row_blocks(p), 152 * 64));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (in_units(p, false)) {
    if (p.dtype == MHLA_BF16)
      launch_units<__nv_bfloat16>(p, false, nullptr, &grid, s);
    else
      launch_units<float>(p, false, nullptr, &grid, s);
  } else if (p.dtype == MHLA_BF16)
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
    const bool any = p.B > 0 && p.Hq + p.Hk > 0;   // the walk over units needs a row
    if (any && in_units(p, true)) {
      if (p.dtype == MHLA_BF16)
        launch_units<__nv_bfloat16>(p, true, part, &grid, s);
      else
        launch_units<float>(p, true, part, &grid, s);
    } else if (p.dtype == MHLA_BF16)
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
