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

constexpr int kBwdBlocks = 608;

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
  if (p.dtype == MHLA_BF16)
    qk_norm_rows<__nv_bfloat16, false><<<grid, 256, 0, s>>>(p, nullptr);
  else
    qk_norm_rows<float, false><<<grid, 256, 0, s>>>(p, nullptr);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int launch_qk_norm_backward(const QkNormProblem& p, void* workspace, void* stream) {
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(row_blocks(p), kBwdBlocks));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* part = static_cast<float*>(workspace);
  {
    KernelTimer timer("qk_norm_backward", stream);
    if (p.dtype == MHLA_BF16)
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
