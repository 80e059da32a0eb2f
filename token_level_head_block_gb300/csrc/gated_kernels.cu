// Gated causal linear attention:
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
// and its gradients.  With dS_t = scale q_t do_t^T + exp(g_{t+1}) dS_{t+1},
//   dq_t = scale S_t do_t         the recurrence itself with (do, v, k) for (q, k, v)
//   dv_t = dS_t^T k_t             the recurrence run backwards with (k, q, do)
//   dk_t = dS_t v_t               the same with (v, do, q)
//   dg_t = exp(g_t) <S_{t-1}, dS_t>, where <S_t, dS_t> = dg_t + k_t . dk_t = dg_{t+1} + q_t . dq_t,
// so dg is a running sum of q . dq - k . dk from the end.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mhla_internal.h"

namespace mhla {
namespace {

constexpr float kLowestGate = -1000.0f;   // exp is 0 in float32 far above this

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

struct Scan {
  Operand q, k, v, g, out, dot;
  const float* init;    // [B][H][d][d] or null
  float* last;          // or null
  float* dots;          // [B][H][N] sums of dot_t . out_t before rounding, or null
  int64_t N, H;
  int32_t d;
  float out_scale, k_scale;
  bool reverse, transposed;   // transposed: init and last hold the state's transpose
};

// One CTA walks one (b, h): thread (c, half) holds half of the state's column c.
template <typename T>
__global__ void __launch_bounds__(256) gated_scan_simple(const Scan a) {
  __shared__ float sq[128], sk[128], sv[128], part[128], red[8];
  const int64_t bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
  const int c = threadIdx.x & 127, r0 = (threadIdx.x >> 7) * 64, d = a.d;
  auto at = [&](const Operand& o, int64_t t) { return static_cast<T*>(o.data) + b * o.sb + t * o.sn + h * o.sh; };
  float S[64];
  for (int i = 0; i < 64; ++i) {
    const int r = r0 + i;
    S[i] = a.init && r < d && c < d ? a.init[bh * d * d + (a.transposed ? c * d + r : r * d + c)] : 0.0f;
  }
  for (int64_t i = 0; i < a.N; ++i) {
    const int64_t t = a.reverse ? a.N - 1 - i : i;
    __syncthreads();
    if (threadIdx.x < 128) {
      sq[c] = c < d ? to_f(at(a.q, t)[c]) : 0.0f;
      sk[c] = c < d ? a.k_scale * to_f(at(a.k, t)[c]) : 0.0f;
      sv[c] = c < d ? to_f(at(a.v, t)[c]) : 0.0f;
    }
    const float decay = expf(fmaxf(to_f(*at(a.g, t)), kLowestGate));
    __syncthreads();
    float o = 0.0f;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      S[j] = fmaf(sk[r0 + j], sv[c], a.reverse ? S[j] : decay * S[j]);
      o = fmaf(sq[r0 + j], S[j], o);
      if (a.reverse) S[j] *= decay;
    }
    if (r0) part[c] = o;
    __syncthreads();
    float dot = 0.0f;
    if (!r0 && c < d) {
      o = a.out_scale * (o + part[c]);
      from_f(at(a.out, t) + c, o);
      if (a.dots) dot = o * to_f(at(a.dot, t)[c]);
    }
    if (a.dots) {
      for (int s = 16; s; s >>= 1) dot += __shfl_xor_sync(~0u, dot, s);
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) a.dots[bh * a.N + t] = red[0] + red[1] + red[2] + red[3];
    }
  }
  if (a.last)
    for (int i = 0; i < 64; ++i) {
      const int r = r0 + i;
      if (r < d && c < d) a.last[bh * d * d + (a.transposed ? c * d + r : r * d + c)] = S[i];
    }
}

// dg of one (b, h): <S, dS> at the end, then the running sum of q.dq - k.dk.
template <typename T>
__global__ void __launch_bounds__(128) gated_gate_grad_simple(const float* qdots, const float* kdots, const float* last,
                                                              const float* dlast, Operand dg, int64_t N, int64_t H,
                                                              int32_t d) {
  __shared__ double red[128];
  const int64_t bh = blockIdx.x, b = bh / H, h = bh % H;
  double s = 0.0;
  if (dlast)
    for (int i = threadIdx.x; i < d * d; i += 128)
      s += static_cast<double>(last[bh * d * d + i]) * static_cast<double>(dlast[bh * d * d + i]);
  red[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 128; ++i) s += red[i];
    for (int64_t t = N - 1; t >= 0; --t) {
      s += static_cast<double>(qdots[bh * N + t]) - static_cast<double>(kdots[bh * N + t]);
      from_f(static_cast<T*>(dg.data) + b * dg.sb + t * dg.sn + h * dg.sh, static_cast<float>(s));
    }
  }
}

Scan scan_of(const GatedProblem& p) {
  Scan a = {};
  a.g = p.g;
  a.N = p.N; a.H = p.H; a.d = p.d;
  a.out_scale = a.k_scale = 1.0f;
  return a;
}

int run_scan(const GatedProblem& p, const Scan& a, void* stream) {
  KernelTimer timer("gated_scan", stream);
  const unsigned grid = static_cast<unsigned>(p.B * p.H);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dtype == MHLA_BF16)
    gated_scan_simple<__nv_bfloat16><<<grid, 256, 0, s>>>(a);
  else
    gated_scan_simple<float><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

}  // namespace

size_t gated_workspace_bytes(const GatedProblem&) { return 0; }

size_t gated_bwd_workspace_bytes(const GatedProblem& p) {
  const int64_t bh = p.B * p.H;
  return 2 * align_up(static_cast<size_t>(bh * p.N) * 4) + align_up(static_cast<size_t>(bh * p.d * p.d) * 4);
}

int launch_gated_forward(const GatedProblem& p, const float* state_in, const Operand& out, float* state_out, void*,
                         void* stream) {
  Scan a = scan_of(p);
  a.q = p.q; a.k = p.k; a.v = p.v;
  a.out = out;
  a.init = state_in;
  a.last = state_out;
  a.out_scale = p.scale;
  return run_scan(p, a, stream);
}

int launch_gated_backward(const GatedProblem& p, const GatedBackward& b, void* workspace, void* stream) {
  const int64_t bh = p.B * p.H;
  char* base = static_cast<char*>(workspace);
  float* qdots = reinterpret_cast<float*>(base);
  base += align_up(static_cast<size_t>(bh * p.N) * 4);
  float* kdots = reinterpret_cast<float*>(base);
  base += align_up(static_cast<size_t>(bh * p.N) * 4);
  float* last = reinterpret_cast<float*>(base);
  Scan a = scan_of(p);
  a.q = b.dout; a.k = p.v; a.v = p.k;
  a.out = b.dq; a.dot = p.q; a.dots = qdots;
  a.out_scale = p.scale;
  a.init = b.state_in; a.last = last; a.transposed = true;
  int rc = run_scan(p, a, stream);
  a = scan_of(p);
  a.reverse = true;
  a.k_scale = p.scale;
  a.q = p.k; a.k = p.q; a.v = b.dout;
  a.out = b.dv;
  a.init = b.dstate_out; a.last = b.dstate_in;
  if (rc == MHLA_OK) rc = run_scan(p, a, stream);
  a.q = p.v; a.k = b.dout; a.v = p.q;
  a.out = b.dk; a.dot = p.k; a.dots = kdots;
  a.last = nullptr; a.transposed = true;
  if (rc == MHLA_OK) rc = run_scan(p, a, stream);
  if (rc != MHLA_OK) return rc;
  KernelTimer timer("gated_gate_grad", stream);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.dtype == MHLA_BF16)
    gated_gate_grad_simple<__nv_bfloat16><<<static_cast<unsigned>(bh), 128, 0, s>>>(qdots, kdots, last, b.dstate_out,
                                                                                   b.dg, p.N, p.H, p.d);
  else
    gated_gate_grad_simple<float><<<static_cast<unsigned>(bh), 128, 0, s>>>(qdots, kdots, last, b.dstate_out, b.dg,
                                                                           p.N, p.H, p.d);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int launch_gated_step(const GatedProblem& p, float* state, const Operand& out, void* stream) {
  return launch_gated_forward(p, state, out, state, nullptr, stream);
}

}  // namespace mhla
