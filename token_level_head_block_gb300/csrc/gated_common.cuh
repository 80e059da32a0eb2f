// What the kernels of the gated recurrence share: the description of a scan, sums of
// log decays, and float32 values as sums of bf16 terms.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "float_pairs.cuh"
#include "mhla_internal.h"

namespace mhla {
namespace gated {

constexpr float kLowestGate = -1000.0f;   // exp is 0 in float32 far above this
constexpr int kSms = 152;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// One scan.  States are [r][c], r of k's channels, c of v's.
struct Scan {
  Operand q, k, v, out, dot;
  const float* init;    // state entering a span, or null for zero
  float* last;          // state after the last span [B][H][d][d], or null
  float* local;         // gated_span_state: a span's own contribution [B][H][spans][d][d]
  float* decay;         // and its decay [B][H][spans]
  float* dots;          // dot_t . (what out_t takes from the state that enters its chunk) [slices][B][H][N], or null
  float* entries;       // the state that enters each chunk [B][H][chunks], as the kernel's threads hold it, or null
  float* sums;          // the running sums of the gates of each chunk, high parts and low parts, or null (forwards)
  float out_scale;      // of the scores
  float state_scale;    // of what a query reads from the state
  float k_scale;        // of what a token adds to the state
  int32_t reverse;
  int32_t init_transposed;
  int32_t init_spans;   // spans per (b, h) in init: slot of a span, or 1
  int32_t join;         // init enters the sequence; local and decay hold what the spans add (tcgen05, forwards)
};

struct ScanSet {
  Scan scan[3];
  Operand g;
  int64_t N, H, BH;
  int64_t span_chunks, chunks;
  int32_t spans, d;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float low(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// A pair as sums of NT bf16 terms, packed.
template <int NT>
__device__ __forceinline__ void split(Two a, uint32_t (&t)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    float x, y;
    apart(a, x, y);
    t[i] = pack(x, y);
    if (i + 1 < NT) a = fma(two(low(t[i]), high(t[i])), two(-1.0f, -1.0f), a);
  }
}
template <int NT>
__device__ __forceinline__ void split(float x, float y, uint32_t (&t)[NT]) {
  split<NT>(two(x, y), t);
}

// A sum of log decays (in powers of two) as the sum of two floats: differences of
// far sums keep the precision of the near ones.
struct Sum {
  float hi, lo;
};
__device__ __forceinline__ Sum add(Sum a, Sum b) {
  const float s = a.hi + b.hi, z = s - a.hi;
  const float e = ((a.hi - (s - z)) + (b.hi - z)) + (a.lo + b.lo);
  Sum r;
  r.hi = s + e;
  r.lo = e - (r.hi - s);
  return r;
}
__device__ __forceinline__ Sum gate_sum(float g) {
  constexpr float kL = 1.4426950408889634f, kLlo = static_cast<float>(1.4426950408889634 - kL);
  g = g < kLowestGate ? kLowestGate : g;   // NaN stays
  Sum r;
  r.hi = g * kL;
  r.lo = fmaf(g, kLlo, fmaf(g, kL, -r.hi));
  return r;
}

__device__ __forceinline__ float exp2_of(Sum a, Sum b) { return exp2_fast((a.hi - b.hi) + (a.lo - b.lo)); }

// Spans a sequence is cut into.
struct Cut {
  int64_t chunks, span_chunks, spans;
};

// tcgen05 kernels (gated_tc_kernels.cu): chunks of 128 tokens, bf16, d <= 64.
constexpr int kTcChunk = 128;
bool tc_supported(const GatedProblem& p);   // by type and size alone
Cut tc_cut(const GatedProblem& p, int scans);
// The tensor maps of a call's scans; false when an operand's address or strides do not suit them.
struct TcMaps {
  CUtensorMap q[3], k[3], v[3];
};
bool tc_maps(const GatedProblem& p, const ScanSet& set, int scans, TcMaps* maps);
int launch_tc_scan(const ScanSet& set, const TcMaps& maps, int scans, bool span_state, cudaStream_t s);

}  // namespace gated
}  // namespace mhla
