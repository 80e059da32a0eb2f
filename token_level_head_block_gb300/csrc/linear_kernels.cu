// A linear layer with its activation and residual, and its gradients:
//   out = act(z) + residual,  z = x w^T + bias         x [rows][k], w [n][k]
//   dz = dout act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum of dz's rows
// All three products are one kernel, linear_gemm, C [M][N] = A B over tcgen05:
//   out   A = x    [M][K]     B = w  [N][K]
//   dx    A = dz   [M][K]     B = w  [K][N]   (read as it lies: N-major)
//   dw    A = dz   [K][M]     B = x  [K][N]   (both read as they lie)
// bf16 matrices whose rows are a multiple of 16 bytes go to TMA as they are.  Others, and float32 ones, are laid out
// first (linear_planes): rows padded to 16 bytes, float32 as the sum of three bf16 terms (2^-24), of whose products the six
// that are not below 2^-24 are formed.  The tensor core truncates what it adds to an accumulator, so float32 keeps
// its small products apart and its large ones in three accumulators, a third of K each, added in the epilogue.
//
// A persistent CTA (or a pair of them with one tile of 256 rows, cta_group::2) loads with TMA, multiplies and finishes the tile before
// at once.  Measured, bf16, against the measured 1947 TFLOP/s and 6.7 TB/s:
//   16384 x 768 by 2304: 44 us, with bias, SiLU and z kept 56 (30 us of products; 27 of HBM's time); 4096 for 768: 168 (159 of products), 0.30 us a
//     chunk of 64 where the products need 0.27; 64 for 768: 24, the finish and HBM (12).  One thread issues a chunk's copies, another its
//     products: with descriptors formed anew for each product it took 0.38 us a chunk whatever the tile (57 us), with two copies a chunk
//     for N-major operands dx and dw took 49 and 60 us for 46 and 53.  Six stages for five were no faster.
//   The finish: rows staged as bf16 and copied out asynchronously; through float32 and ordinary stores 60 us for 56, 35 for 24.
//   262144 x 384 by 384 with residual: 114 us (91 of HBM's time); 126 when the next tile's residual is not asked for as far as L2, 117 for the
//     one after it; ordinary stores, since the residual is read as it lies.
//
// Few rows (serving) read w once and compute next to nothing: linear_rows gives every CTA 16 of w's rows and
// its warps a part of K each.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "gated_common.cuh"
#include "mhla_internal.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma_host.h"
#include "warp_mma.cuh"

namespace mhla {

__device__ unsigned int g_linear_error = 0;

namespace {

using namespace ptx;
using namespace tc;

using gated::from_f;
using gated::low;
using gated::high;
using gated::to_f;

// ----------------------------------------------------------------- activations

// 1 + e^-z; FAST for results that are rounded to bf16 (2^-8; ex2 and the reciprocal are good to 2^-21; a quotient by 2^126 or
// more is 0).
template <bool FAST>
__device__ __forceinline__ float over_sigmoid(float z) { return 1.0f + (FAST ? __expf(-z) : expf(-z)); }

constexpr float kTanhScale = 0.7978845608028654f, kTanhCube = 0.044715f;   // sqrt(2 / pi)

// Phi(z) = erfc(-z / sqrt 2) / 2; (1 + erf(z / sqrt 2)) / 2 cancels for z < 0, 4% off at -5.  FAST: Phi(-s) = e^(-s^2 / 2) P(t), t = 1 / (1 +
// 0.265 s), P a polynomial without a constant term fitted to the quotient over [0, 15] for the least relative error (Remez's criterion by reweighted
// least squares in 64 bits), 2^-20; behind that the exponential is 0.  `e` receives e^(-z^2 / 2).  [16384, 768] x 2304, z kept, and
// its gradients, called: erff 70 and 173 us, erfcf 97 and 200, this 71 and 161; float32 erff 315 and 700, erfcf 348 and 722.
template <bool FAST>
__device__ __forceinline__ float normal_below(float z, float& e) {
  e = FAST ? __expf(-0.5f * z * z) : expf(-0.5f * z * z);
  if (!FAST) return 0.5f * erfcf(z * -0.7071067811865476f);
  const float t = __fdividef(1.0f, fmaf(0.265f, fabsf(z), 1.0f));
  float p = fmaf(-0.067709036f, t, 0.195002005f);
  p = fmaf(p, t, -0.065985590f);
  p = fmaf(p, t, 0.142225206f);
  p = fmaf(p, t, 0.083048776f);
  p = fmaf(p, t, 0.107817046f);
  p = fmaf(p, t, 0.105601341f);
  const float q = p * t * e;
  return z < 0.0f ? q : 1.0f - q;
}

template <bool FAST, int ACT>
__device__ __forceinline__ float activate(float z) {
  if (ACT == MHLA_ACT_RELU) return z < 0.0f ? 0.0f : z;   // NaN stays
  if (ACT == MHLA_ACT_GELU) {
    float e;
    return z * normal_below<FAST>(z, e);
  }
  if (ACT == MHLA_ACT_GELU_TANH) {   // (1 + tanh u) / 2 = 1 / (1 + e^-2u)
    const float u = kTanhScale * fmaf(kTanhCube * z * z, z, z);
    return FAST ? __fdividef(z, over_sigmoid<true>(2.0f * u)) : z / over_sigmoid<false>(2.0f * u);
  }
  if (ACT == MHLA_ACT_SILU) return FAST ? __fdividef(z, over_sigmoid<true>(z)) : z / over_sigmoid<false>(z);
  return z;
}

// One branch for all of them, so that each activation's code stands once.
template <bool FAST, int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
  auto all = [&](auto one) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = one(z[i]);
  };
  switch (act) {
    case MHLA_ACT_RELU: all([](float x) { return activate<FAST, MHLA_ACT_RELU>(x); }); break;
    case MHLA_ACT_GELU: all([](float x) { return activate<FAST, MHLA_ACT_GELU>(x); }); break;
    case MHLA_ACT_GELU_TANH: all([](float x) { return activate<FAST, MHLA_ACT_GELU_TANH>(x); }); break;
    case MHLA_ACT_SILU: all([](float x) { return activate<FAST, MHLA_ACT_SILU>(x); }); break;
    default: break;
  }
}

template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) { return FAST ? __fdividef(1.0f, over_sigmoid<true>(z)) : 1.0f / over_sigmoid<false>(z); }

template <bool FAST, int ACT>
__device__ __forceinline__ float slope(float z) {
  if (ACT == MHLA_ACT_RELU) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
  if (ACT == MHLA_ACT_GELU) {
    float e;
    const float below = normal_below<FAST>(z, e);
    return fmaf(z * 0.3989422804014327f, e, below);
  }
  if (ACT == MHLA_ACT_GELU_TANH) {
    z = z > 30.0f ? 30.0f : z < -30.0f ? -30.0f : z;   // 1 and 0 there; the cube stays finite
    const float u = kTanhScale * fmaf(kTanhCube * z * z, z, z), p = sigmoid<FAST>(2.0f * u);
    return p + z * p * (1.0f - p) * (2.0f * kTanhScale) * fmaf(3.0f * kTanhCube * z, z, 1.0f);
  }
  const float p = sigmoid<FAST>(z);
  return p * fmaf(z, 1.0f - p, 1.0f);
}

// v *= act'(z)
template <bool FAST, int N>
__device__ __forceinline__ void times_slope(float (&v)[N], const float (&z)[N], int act) {
  auto all = [&](auto one) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] *= one(z[i]);
  };
  switch (act) {
    case MHLA_ACT_RELU: all([](float x) { return slope<FAST, MHLA_ACT_RELU>(x); }); break;
    case MHLA_ACT_GELU: all([](float x) { return slope<FAST, MHLA_ACT_GELU>(x); }); break;
    case MHLA_ACT_GELU_TANH: all([](float x) { return slope<FAST, MHLA_ACT_GELU_TANH>(x); }); break;
    default: all([](float x) { return slope<FAST, MHLA_ACT_SILU>(x); }); break;
  }
}

// ----------------------------------------------------------------- epilogue

struct Finish {
  void* out;             // [M][N] of the call's type
  void* pre;             // z, or null
  const void* residual;  // [M][N], or null; may be out
  const void* bias;      // [N], or null
  int64_t M, N;
  int32_t act;
  int32_t quads;         // N % 4 == 0: four values an access
};

template <bool F32>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <bool F32>
__device__ __forceinline__ void store_one(void* p, int64_t i, float x) {
  if (F32)
    static_cast<float*>(p)[i] = x;
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

// Four values as they lie, asked for ahead of their use.
template <bool F32>
struct Quad {
  typename std::conditional<F32, float4, uint2>::type x;
  __device__ __forceinline__ void fetch(const void* p, int64_t i) {
    if constexpr (F32)
      x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    else
      x = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  __device__ __forceinline__ float4 value() const {
    if constexpr (F32)
      return x;
    else
      return make_float4(low(x.x), high(x.x), low(x.y), high(x.y));
  }
  __device__ __forceinline__ void set(float4 v) {
    if constexpr (F32)
      x = v;
    else
      x = make_uint2(gated::pack(v.x, v.y), gated::pack(v.z, v.w));
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    if constexpr (F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = x;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = x;
  }
};

__device__ __forceinline__ float4 plus(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// ROWS times four sums with the bias, those of row r from element i + r step on, N % 4 == 0; rows behind `rows` are left out.
template <bool F32, int ROWS>
__device__ __forceinline__ void finish_quads(const Finish& f, int64_t i, int64_t step, int rows, float (&z)[4 * ROWS],
                                             const Quad<F32> (&residual)[ROWS]) {
  Quad<F32> q;
  if (f.pre)
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (r < rows) {
        q.set(make_float4(z[4 * r], z[4 * r + 1], z[4 * r + 2], z[4 * r + 3]));
        q.store(f.pre, i + r * step);
      }
  activate_all<!F32>(z, f.act);
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (r < rows) {
      float4 y = make_float4(z[4 * r], z[4 * r + 1], z[4 * r + 2], z[4 * r + 3]);
      if (f.residual) y = plus(y, residual[r].value());
      q.set(y);
      q.store(f.out, i + r * step);
    }
}

template <bool F32>
__device__ __forceinline__ float4 bias_quad(const Finish& f, int64_t c) {
  if (!f.bias) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (f.quads) {
    Quad<F32> q;
    q.fetch(f.bias, c);
    return q.value();
  }
  float b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = c + e < f.N ? load_one<F32>(f.bias, c + e) : 0.0f;
  return make_float4(b[0], b[1], b[2], b[3]);
}

// Four sums of row r, columns c .. c + 3 (r < M, c < N), any N.
template <bool F32>
__device__ __forceinline__ void finish_quad(const Finish& f, int64_t r, int64_t c, float4 z) {
  const int64_t i = r * f.N + c;
  z = plus(z, bias_quad<F32>(f, c));
  float zs[4] = {z.x, z.y, z.z, z.w};
  if (f.quads) {
    Quad<F32> s[1] = {};
    if (f.residual) s[0].fetch(f.residual, i);
    finish_quads<F32, 1>(f, i, 0, 1, zs, s);
  } else {
    if (f.pre)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < f.N) store_one<F32>(f.pre, i + e, zs[e]);
    activate_all<!F32>(zs, f.act);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e >= f.N) break;
      store_one<F32>(f.out, i + e, f.residual ? zs[e] + load_one<F32>(f.residual, i + e) : zs[e]);
    }
  }
}

// ----------------------------------------------------------------- product

struct Product {
  CUtensorMap a, b, out, pre;   // out, pre: of bulk stores
  Finish f;
  float* parts;          // [splits][M][pitch] sums of parts of K, or null
  int64_t pitch, units;
  int32_t a_major, b_major;   // 1: the operand lies [K][M] ([K][N])
  int32_t a_blocks, b_blocks; // and one copy takes all its blocks of 64 columns
  int32_t BN, tiles_n, chunks, splits, split_chunks;
};

// PAIR: two CTAs with one tile of 256 rows (cta_group::2), each loading its rows of A and half of B's.
template <int TERMS, bool PAIR>
struct GemmLay {
  static constexpr int BM = 128, BK = 64;                // rows of a CTA
  static constexpr int MOST_N = TERMS == 1 ? 256 : 128;
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = MOST_N / (PAIR ? 2 : 1) * BK * 2;
  static constexpr int STAGE = TERMS * (A_BYTES + B_BYTES), NS = PAIR ? 5 : TERMS == 1 ? 4 : 2;
  static constexpr int ACCS = TERMS == 1 ? 2 : 1;        // tiles whose sums tensor memory holds
  static constexpr int MAINS = TERMS == 1 ? 1 : 3;       // accumulators of the large products
  static constexpr int GROUP = PAIR ? 32 : 16;           // columns a warp finishes at once
  static constexpr int PITCH = GROUP + 4, STAGING = 32 * PITCH * 4;   // a warp's 32 rows of them
  static constexpr int SIDE = PAIR ? 3 : 2;              // finishing warps beside one another
  static constexpr int WARPS = 4 * SIDE, THREADS = 64 + 32 * WARPS;
  static constexpr size_t SMEM = static_cast<size_t>(NS) * STAGE + WARPS * STAGING + 1024 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(!PAIR || (GROUP == 32 && STAGING % 512 == 0 && STAGING >= 4096), "bulk stores' staging");
};

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_bounded_on(bar, parity, abort_flag, &g_linear_error);   // the first look without a call
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return warp_wait_on(bar, parity, abort_flag, &g_linear_error);
}
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) { drain_wait_on(bar, parity, &g_linear_error); }

// Unit u: a tile and a part of K.
struct Unit {
  int32_t m0, n0, first, count, split;
};
template <bool PAIR>
__device__ __forceinline__ Unit unit_of(const Product& p, int64_t u, uint32_t rank) {
  Unit r;
  r.split = static_cast<int32_t>(u % p.splits);
  const int64_t t = u / p.splits;
  r.n0 = static_cast<int32_t>(t % p.tiles_n) * p.BN;
  r.m0 = static_cast<int32_t>(t / p.tiles_n) * (PAIR ? 256 : 128) + (PAIR ? 128 * static_cast<int32_t>(rank) : 0);
  r.first = r.split * p.split_chunks;
  r.count = min(p.split_chunks, p.chunks - r.first);
  return r;
}

// Persistent CTAs walk the units, neighbours sharing A's rows in L2.  Warp 0 loads K chunks of 64 (a ring of
// stages), warp 1 issues the MMAs, eight warps turn the sums round through shared memory, so that a row's columns lie in
// neighbouring lanes, and finish them.
// BULK: finished rows leave through the copy engine.
template <int TERMS, bool PAIR, bool BULK>
__global__ void __launch_bounds__(GemmLay<TERMS, PAIR>::THREADS, 1) linear_gemm(const __grid_constant__ Product p) {
  using L = GemmLay<TERMS, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint8_t* staging = smem + L::NS * L::STAGE;
  uint8_t* ctrl = staging + L::WARPS * L::STAGING;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + L::NS;
  uint64_t* tfull = empty + L::NS;
  uint64_t* tempty = tfull + 2;
  uint64_t* fin = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 512);
  volatile uint32_t* abortf = tmem_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::NS; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tempty + a, (PAIR ? 2 : 1) * L::WARPS);   // one arrival a warp
    }
    mbar_init(fin, 1);
    *abortf = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.a);
    prefetch_tmap(&p.b);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync();   // both CTAs' barriers and tensor memory are there
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int64_t first_unit = PAIR ? blockIdx.x / 2 : blockIdx.x, stride = PAIR ? gridDim.x / 2 : gridDim.x;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t policy = policy_evict_last();
      int s = 0;
      uint32_t ph = 0;
      uint64_t fills = 0;
      bool ok = true;
      const int b_rows = PAIR ? p.BN / 2 : p.BN;
      const uint32_t bytes = TERMS * (L::A_BYTES + b_rows * L::BK * 2);
      const uint32_t full_of_0 = PAIR ? address_at(full, 0) : 0u;   // rank 0's barriers count both CTAs' bytes
      auto load = [&](uint8_t* at, const CUtensorMap* map, int st, int32_t x, int32_t y, int32_t z) {
        if (PAIR)
          tma_load_3d_pair(at, map, full_of_0 + 8 * st, x, y, z, policy);
        else
          tma_load_3d(at, map, full + st, x, y, z, policy);
      };
      for (int64_t u = first_unit; ok && u < p.units; u += stride) {
        const Unit un = unit_of<PAIR>(p, u, rank);
        const int32_t n0 = un.n0 + static_cast<int32_t>(rank) * b_rows;
        for (int kc = 0; kc < un.count; ++kc) {
          if (!wait_bounded(empty + s, ph ^ 1u, abortf)) { ok = false; break; }
          if (rank == 0) mbar_arrive_expect_tx(full + s, (PAIR ? 2 : 1) * bytes);
          uint8_t* st = smem + s * L::STAGE;
          const int32_t k0 = (un.first + kc) * L::BK;
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            uint8_t* at = st + t * L::A_BYTES;
            if (TERMS == 1 && p.a_blocks) {
              load(at, &p.a, s, 0, k0, un.m0 / 64);
            } else if (p.a_major) {
              load(at, &p.a, s, un.m0, k0, t);
              load(at + 8192, &p.a, s, un.m0 + 64, k0, t);
            } else {
              load(at, &p.a, s, k0, un.m0, t);
            }
            at = st + TERMS * L::A_BYTES + t * L::B_BYTES;
            if (TERMS == 1 && p.b_blocks) {
              load(at, &p.b, s, 0, k0, n0 / 64);
            } else if (p.b_major) {
              for (int j = 0; j < b_rows / 64; ++j) load(at + 8192 * j, &p.b, s, n0 + 64 * j, k0, t);
            } else {
              load(at, &p.b, s, k0, n0, t);
            }
          }
          ++fills;
          if (++s == L::NS) { s = 0; ph ^= 1u; }
        }
      }
      if (rank == 0)
        for (int st = 0; st < L::NS; ++st) {
          const uint64_t n = fills / L::NS + (static_cast<uint64_t>(st) < fills % L::NS ? 1 : 0);
          if (n > 0) drain_wait(full + st, static_cast<uint32_t>((n - 1) & 1));
        }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(PAIR ? 256 : 128, p.BN, p.a_major != 0, p.b_major != 0);
      // steps of 16 of K: 32 bytes along swizzled rows, or 16 rows of 128 bytes
      // One thread issues everything, so what it computes in between is kept short: descriptors of the first stage, to whose address
      // fields (units of 16 bytes, below 2^14 over all of shared memory) the rest is added.
      const uint32_t a_step = (p.a_major ? 2048 : 32) / 16, b_step = (p.b_major ? 2048 : 32) / 16;
      const uint64_t a_first = smem_desc(smem_u32(smem), p.a_major ? 8192 : 16, 1024, 2);
      const uint64_t b_first = smem_desc(smem_u32(smem) + TERMS * L::A_BYTES, p.b_major ? 8192 : 16, 1024, 2);
      auto commit = [&](uint64_t* bar) {
        if (PAIR)
          mma_commit_pair(bar);
        else
          mma_commit(bar);
      };
      int s = 0;
      uint32_t ph = 0, local = 0;
      bool ok = true;
      for (int64_t u = first_unit; ok && u < p.units; u += stride, ++local) {
        const Unit un = unit_of<PAIR>(p, u, rank);
        const uint32_t acc = local % L::ACCS, aph = (local / L::ACCS) & 1u;
        if (!wait_bounded(tempty + acc, aph ^ 1u, abortf)) break;
        tc_fence_after();
        const uint32_t dt = tmem + acc * 256;
        for (int kc = 0; kc < un.count; ++kc) {
          if (!wait_bounded(full + s, ph, abortf)) { ok = false; break; }
          tc_fence_after();
          const uint64_t a_stage = a_first + s * (L::STAGE / 16), b_stage = b_first + s * (L::STAGE / 16);
          // the accumulator of this part of K, and whether it is empty yet
          const int main = L::MAINS == 1 ? 0 : L::MAINS * kc / un.count;
          const bool opens = L::MAINS == 1 ? kc == 0 : kc == (main * un.count + L::MAINS - 1) / L::MAINS;
#pragma unroll
          for (int ks = 0; ks < L::BK / 16; ++ks)
#pragma unroll
            for (int i = TERMS - 1; i >= 0; --i)
#pragma unroll
              for (int j = TERMS - 1 - i; j >= 0; --j) {
                const bool large = i + j == 0;
                const uint64_t a = a_stage + (i * (L::A_BYTES / 16) + ks * a_step), b = b_stage + (j * (L::B_BYTES / 16) + ks * b_step);
                const bool first = large ? opens && ks == 0 : kc == 0 && ks == 0 && i == TERMS - 1;
                const uint32_t to = dt + (large ? 128 * main : 128 * L::MAINS);
                if (PAIR)
                  mma_bf16_pair(to, a, b, idesc, first ? 0u : 1u);
                else
                  mma_bf16(to, a, b, idesc, first ? 0u : 1u);
              }
          commit(empty + s);
          if (++s == L::NS) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        commit(tfull + acc);
      }
      commit(fin);
      drain_wait(fin, 0);
    }
  } else {
    const int q4 = warp & 3, side = (warp - 2) >> 2;   // TMEM lane quarter this warp may read; every SIDE-th group of columns is its own
    float* stage = reinterpret_cast<float*>(staging + (warp - 2) * L::STAGING);
    constexpr bool F32 = TERMS > 1;
    constexpr int GROUP = L::GROUP, LANES = GROUP / 4, STEP = 32 / LANES, ROWS = 32 / STEP;   // lanes a row, rows at once, rows a lane
    const bool whole = p.f.quads && !p.parts;
    const int lane_row = lane / LANES, lane_col = 4 * (lane % LANES);
    uint32_t local = 0;
    for (int64_t u = first_unit; u < p.units; u += stride, ++local) {
      const Unit un = unit_of<PAIR>(p, u, rank);
      const uint32_t acc = local % L::ACCS, aph = (local / L::ACCS) & 1u;
      const int64_t row0 = un.m0 + 32 * q4 + lane_row, c0 = un.n0 + lane_col;
      const int64_t i0 = row0 * p.f.N + c0;
      const int rows = static_cast<int>(max(int64_t{0}, min(int64_t{ROWS}, (p.f.M - row0 + STEP - 1) / STEP)));   // of this lane's
      // what the finish reads of memory: the first group's while the products run, then a group ahead
      Quad<F32> residual[ROWS] = {}, bias = {};
      auto fetch = [&](int gi) {
        if (BULK || !whole || c0 + GROUP * gi >= p.f.N) return;
        if (p.f.bias) bias.fetch(p.f.bias, c0 + GROUP * gi);
        if (p.f.residual)
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            if (i < rows) residual[i].fetch(p.f.residual, i0 + STEP * i * p.f.N + GROUP * gi);
      };
      fetch(side);
      if (whole && p.f.residual && u + stride < p.units) {   // the next tile's, as far as L2
        const Unit next = unit_of<PAIR>(p, u + stride, rank);
        const int64_t row = next.m0 + 32 * q4 + lane;
        if (row < p.f.M)
          for (int64_t c = next.n0 + GROUP * side; c < min(p.f.N, next.n0 + static_cast<int64_t>(p.BN)); c += GROUP * L::SIDE)
            prefetch_l2(static_cast<const char*>(p.f.residual) + (row * p.f.N + c) * (F32 ? 4 : 2));
      }
      if (!warp_wait(tfull + acc, aph, abortf)) break;
      tc_fence_after();
      const uint32_t tb = tmem + acc * 256 + (static_cast<uint32_t>(32 * q4) << 16);
      const int mains = TERMS == 1 ? 1 : min(un.count, L::MAINS);
      const int used = static_cast<int>(min(static_cast<int64_t>(p.BN / GROUP), (p.f.N - un.n0 + GROUP - 1) / GROUP));
#pragma unroll 1
      for (int gi = side; gi < used; gi += L::SIDE) {
        uint32_t v[GROUP];
        if constexpr (TERMS > 1) {
          uint32_t x[16], y[16], z[16];
          tmem_ld_x16(tb + 16 * gi, v);
          tmem_ld_x16(tb + 128 * L::MAINS + 16 * gi, z);
          if (mains > 1) tmem_ld_x16(tb + 128 + 16 * gi, x);
          if (mains > 2) tmem_ld_x16(tb + 256 + 16 * gi, y);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float sum = __uint_as_float(z[e]);
            if (mains > 2) sum += __uint_as_float(y[e]);
            if (mains > 1) sum += __uint_as_float(x[e]);
            v[e] = __float_as_uint(__uint_as_float(v[e]) + sum);
          }
        } else {
          if constexpr (GROUP == 32)
            tmem_ld_x32(tb + 32 * gi, v);
          else
            tmem_ld_x16(tb + 16 * gi, v);
          tmem_ld_wait();
        }
        float z[4 * ROWS];
        if constexpr (BULK) {
          // a lane keeps its row of the group: bf16 rows staged as the copies take them, 16-byte units changing places with the row
          const int64_t c = un.n0 + GROUP * gi;
#pragma unroll
          for (int j = 0; j < GROUP / 8; ++j) {
            uint4 add = make_uint4(0u, 0u, 0u, 0u);
            if (p.f.bias && c + 8 * j < p.f.N) add = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.f.bias) + c + 8 * j));
            const uint32_t adds[4] = {add.x, add.y, add.z, add.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              z[8 * j + 2 * i] = __uint_as_float(v[8 * j + 2 * i]) + low(adds[i]);
              z[8 * j + 2 * i + 1] = __uint_as_float(v[8 * j + 2 * i + 1]) + high(adds[i]);
            }
          }
          if (lane == 0) bulk_wait_group_read0();   // what the copies before read
          __syncwarp();
          auto put = [&](int where) {
#pragma unroll
            for (int j = 0; j < GROUP / 8; ++j)
              *reinterpret_cast<uint4*>(reinterpret_cast<char*>(stage) + where + 64 * lane + ((j ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(gated::pack(z[8 * j], z[8 * j + 1]), gated::pack(z[8 * j + 2], z[8 * j + 3]), gated::pack(z[8 * j + 4], z[8 * j + 5]),
                             gated::pack(z[8 * j + 6], z[8 * j + 7]));
          };
          if (p.f.pre) put(2048);
          activate_all<true>(z, p.f.act);
          put(0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int32_t row = un.m0 + 32 * q4;
            if (row < p.f.M) {
              tma_store_2d(&p.out, stage, static_cast<int32_t>(c), row);
              if (p.f.pre) tma_store_2d(&p.pre, reinterpret_cast<char*>(stage) + 2048, static_cast<int32_t>(c), row);
              bulk_commit_group();
            }
          }
        } else {
          // a row of the group a lane becomes four columns of ROWS rows
#pragma unroll
          for (int e = 0; e < LANES; ++e)
            *reinterpret_cast<uint4*>(stage + lane * L::PITCH + 4 * e) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          __syncwarp();
          const float4 add = p.f.bias ? bias.value() : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < ROWS; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(stage + (STEP * i + lane_row) * L::PITCH + lane_col);
            z[4 * i] = x.x; z[4 * i + 1] = x.y; z[4 * i + 2] = x.z; z[4 * i + 3] = x.w;
          }
          __syncwarp();
          const int64_t c = c0 + GROUP * gi;
          if (whole) {
            Quad<F32> now[ROWS];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
              now[i] = residual[i];
              z[4 * i] += add.x; z[4 * i + 1] += add.y; z[4 * i + 2] += add.z; z[4 * i + 3] += add.w;
            }
            if (gi + L::SIDE < used) fetch(gi + L::SIDE);
            if (c < p.f.N) finish_quads<F32, ROWS>(p.f, i0 + GROUP * gi, STEP * p.f.N, rows, z, now);
          } else if (c < p.f.N) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
              if (i >= rows) break;
              const float4 x = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
              if (p.parts)
                *reinterpret_cast<float4*>(p.parts + (un.split * p.f.M + row0 + STEP * i) * p.pitch + c) = x;
              else
                finish_quad<F32>(p.f, row0 + STEP * i, c, x);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {   // the sums are read out
        if (PAIR)
          mbar_arrive_at(tempty + acc, 0);
        else
          mbar_arrive(tempty + acc);
      }
    }
  }
  if (BULK && warp > 1 && lane == 0) bulk_wait_group0();
  tc_fence_before();
  // neither CTA leaves while the other's MMAs read its shared memory or their commits arrive there
  __syncthreads();
  if (PAIR) {
    if (rank == 1 && threadIdx.x == 32) drain_wait(fin, 0);   // the last of rank 0's commits, behind those this CTA waited for
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

// Sums of the parts of K, finished.
struct Join {
  Finish f;
  const float* parts;
  int64_t pitch;
  int32_t splits;
};
template <bool F32>
__global__ void __launch_bounds__(256) linear_join(const __grid_constant__ Join p) {
  const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x), total = p.f.M * p.pitch;
  if (i >= total) return;
  const int64_t r = i / p.pitch, c = i % p.pitch;
  if (c >= p.f.N) return;
  float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < p.splits; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(p.parts + s * total + i);
    z.x += x.x; z.y += x.y; z.z += x.z; z.w += x.w;
  }
  finish_quad<F32>(p.f, r, c, z);
}

// ----------------------------------------------------------------- planes

// [rows][cols] as TERMS planes of bf16 rows `pitch` apart; with `pre`, times the activation's slope there.  Column sums
// of what is laid out (in float32) by blocks of rows to `sums` [blocks][cols], or null; dst null: the sums alone.
struct Planes {
  const void* src;
  const void* pre;
  __nv_bfloat16* dst;
  float* sums;
  int64_t rows, cols, pitch, block_rows;
  int32_t act;
};

// Up to three matrices at once: a launch costs more than a small one of them.
struct PlaneSet {
  Planes of[3];
};

// A thread has VEC columns; 32 threads side by side, eight rows at once.
template <int TERMS, int VEC>
__global__ void __launch_bounds__(256) linear_planes(const __grid_constant__ PlaneSet set) {
  __shared__ float part[8][32 * VEC];
  const Planes& p = set.of[blockIdx.z];
  if (static_cast<int64_t>(blockIdx.x) * 32 * VEC >= p.cols || blockIdx.y * p.block_rows >= p.rows) return;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + x) * VEC;
  const int64_t first = blockIdx.y * p.block_rows, last = min(p.rows, first + p.block_rows);
  float sum[VEC] = {};
  constexpr int BATCH = 4;   // rows in flight
  using Wide = typename std::conditional<VEC == 8, uint4, typename std::conditional<VEC == 4, uint4, uint32_t>::type>::type;
  auto fetch = [&](const void* q, int64_t i) {
    Wide x;
    if constexpr (VEC == 1)
      x = __float_as_uint(load_one<(TERMS > 1)>(q, i));
    else if constexpr (TERMS > 1)
      x = *reinterpret_cast<const uint4*>(static_cast<const float*>(q) + i);
    else
      x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(q) + i);
    return x;
  };
  auto open = [&](const Wide& x, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      v[0] = __uint_as_float(x);
    } else if constexpr (VEC == 4) {
      v[0] = __uint_as_float(x.x); v[1] = __uint_as_float(x.y); v[2] = __uint_as_float(x.z); v[3] = __uint_as_float(x.w);
    } else {
      v[0] = low(x.x); v[1] = high(x.x); v[2] = low(x.y); v[3] = high(x.y);
      v[4] = low(x.z); v[5] = high(x.z); v[6] = low(x.w); v[7] = high(x.w);
    }
  };
  if (c < p.cols) {
    for (int64_t r0 = first + y; r0 < last; r0 += 8 * BATCH) {
      Wide a[BATCH], w[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)
        if (r0 + 8 * j < last) {
          a[j] = fetch(p.src, (r0 + 8 * j) * p.cols + c);
          if (p.pre) w[j] = fetch(p.pre, (r0 + 8 * j) * p.cols + c);
        }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {   // one branch an activation: the rest of the code is small
        const int64_t r = r0 + 8 * j;
        if (r >= last) break;
        float v[VEC], z[VEC];
        open(a[j], v);
        if (p.pre) {
          open(w[j], z);
          times_slope<TERMS == 1>(v, z, p.act);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] += v[e];
        if (!p.dst) continue;
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          __nv_bfloat16* to = p.dst + (t * p.rows + r) * p.pitch + c;
          float h[VEC];
#pragma unroll
          for (int e = 0; e < VEC; ++e) h[e] = __bfloat162float(__float2bfloat16_rn(v[e]));
          if constexpr (VEC == 8)
            *reinterpret_cast<uint4*>(to) = make_uint4(gated::pack(h[0], h[1]), gated::pack(h[2], h[3]), gated::pack(h[4], h[5]), gated::pack(h[6], h[7]));
          else if constexpr (VEC == 4)
            *reinterpret_cast<uint2*>(to) = make_uint2(gated::pack(h[0], h[1]), gated::pack(h[2], h[3]));
          else
            from_f(to, h[0]);
          // an infinity is its first term alone
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[e] = fabsf(h[e]) < __int_as_float(0x7F800000) ? v[e] - h[e] : 0.0f;
        }
      }
    }
  }
  if (!p.sums) return;
#pragma unroll
  for (int e = 0; e < VEC; ++e) part[y][x * VEC + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * VEC; i += 256) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * VEC + i;
    if (col >= p.cols) continue;
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += part[j][i];
    p.sums[blockIdx.y * p.cols + col] = s;
  }
}

// Column sums of the blocks, in their order: one warp a column.
template <bool F32>
__global__ void __launch_bounds__(256) linear_column_sums(const float* sums, void* out, int64_t cols, int32_t blocks) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (c >= cols) return;
  const int lane = threadIdx.x & 31;
  float s = 0.0f;
  for (int b = lane; b < blocks; b += 32) s += sums[b * cols + c];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  if (lane == 0) store_one<F32>(out, c, s);
}

// ----------------------------------------------------------------- few rows

// 16 of w's rows and ROWS (a multiple of 8) of x's.  Each of eight warps takes every eighth step of K and holds its operands straight from
// memory: a lane's 16 bytes of a row are k = 8 (lane % 4) .. + 7 of a step of 32, and enter two MMAs as the k that its
// place stands for; w and x agree on which, so the sum is the same.
template <int GROUPS>   // of eight rows
__global__ void __launch_bounds__(256) linear_rows(const __nv_bfloat16* x, const __nv_bfloat16* w, int64_t rows, int32_t k, const Finish f) {
  __shared__ float part[8][16][8 * GROUPS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16, r0 = static_cast<int64_t>(blockIdx.y) * 8 * GROUPS;
  float acc[GROUPS][4] = {};
  const __nv_bfloat16 *w0 = w + (n0 + g) * k + 8 * t, *w1 = w0 + 8 * static_cast<int64_t>(k);
  const bool in0 = n0 + g < f.N, in1 = n0 + g + 8 < f.N;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
  for (int k0 = 32 * warp; k0 < k; k0 += 256) {
    const bool in = k0 + 8 * t < k;   // k % 8 == 0
    const uint4 a0 = in && in0 ? __ldg(reinterpret_cast<const uint4*>(w0 + k0)) : none;
    const uint4 a1 = in && in1 ? __ldg(reinterpret_cast<const uint4*>(w1 + k0)) : none;
    const uint32_t first[4] = {a0.x, a1.x, a0.y, a1.y}, second[4] = {a0.z, a1.z, a0.w, a1.w};
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      const int64_t r = r0 + 8 * i + g;
      const uint4 b = in && r < rows ? __ldg(reinterpret_cast<const uint4*>(x + r * k + k0 + 8 * t)) : none;
      gated::mma(acc[i], first, b.x, b.y);
      gated::mma(acc[i], second, b.z, b.w);
    }
  }
#pragma unroll
  for (int i = 0; i < GROUPS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[warp][g + 8 * (e >> 1)][8 * i + 2 * t + (e & 1)] = acc[i][e];
  __syncthreads();
  for (int i = threadIdx.x; i < 4 * 8 * GROUPS; i += 256) {
    const int r = i / 4, c = 4 * (i % 4);
    if (r0 + r >= rows || n0 + c >= f.N) continue;
    float z[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[e] += part[j][c + e][r];
    finish_quad<false>(f, r0 + r, n0 + c, make_float4(z[0], z[1], z[2], z[3]));
  }
}

// Float32 and rows that 16-byte loads do not take: a warp has one of w's rows and eight of x's.
template <typename T>
__global__ void __launch_bounds__(256) linear_dots(const T* x, const T* w, int64_t rows, int32_t k, const Finish f) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5), r0 = static_cast<int64_t>(blockIdx.y) * 8;
  const int lane = threadIdx.x & 31;
  if (n >= f.N) return;
  float acc[8] = {};
  const int m = static_cast<int>(min(rows - r0, int64_t{8}));
#pragma unroll 4
  for (int i = lane; i < k; i += 32) {
    const float a = to_f(w[n * k + i]);
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < m) acc[r] = fmaf(a, to_f(x[(r0 + r) * k + i]), acc[r]);
  }
  float mine = 0.0f;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[r] += __shfl_xor_sync(~0u, acc[r], o);
    if (lane == r) mine = acc[r];
  }
  if (lane >= m) return;
  const int64_t i = (r0 + lane) * f.N + n;
  constexpr bool F32 = sizeof(T) == 4;
  const float z = mine + (f.bias ? load_one<F32>(f.bias, n) : 0.0f);
  if (f.pre) store_one<F32>(f.pre, i, z);
  float y[1] = {z};
  activate_all<!F32>(y, f.act);
  store_one<F32>(f.out, i, f.residual ? y[0] + load_one<F32>(f.residual, i) : y[0]);
}

// ----------------------------------------------------------------- host

constexpr int kSms = 152;

struct Matrix {          // [terms][rows][pitch] of bf16, cols of them used
  const void* data;
  int64_t rows, cols, pitch;
};

bool direct(int64_t cols, int dtype) { return dtype == MHLA_BF16 && cols % 8 == 0; }
int64_t plane_pitch(int64_t cols) { return (cols + 7) / 8 * 8; }
size_t plane_bytes(int64_t rows, int64_t cols, int dtype) {
  return align_up(static_cast<size_t>(rows * plane_pitch(cols)) * 2 * (dtype == MHLA_BF16 ? 1 : 3));
}

bool encode_planes(CUtensorMap* m, const Matrix& x, int terms, int box_cols, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(x.cols), static_cast<cuuint64_t>(x.rows), static_cast<cuuint64_t>(terms)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.pitch * 2), static_cast<cuuint64_t>(x.rows * x.pitch * 2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  return encode_tensor_map(m, 3, const_cast<void*>(x.data), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Columns as blocks of 64 (a whole number of them), `count` a box: where a matrix is read N-major, one copy takes a chunk's.
bool encode_blocks(CUtensorMap* m, const Matrix& x, int count) {
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(x.rows), static_cast<cuuint64_t>(x.cols / 64)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.pitch * 2), 128};
  const cuuint32_t box[3] = {64, 64, static_cast<cuuint32_t>(count)};
  return encode_tensor_map(m, 3, const_cast<void*>(x.data), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// How C [M][N] over K is cut.  Time of a unit: its chunks, by the operand bytes that an SM takes in (a chunk of 128 + 256 rows is
// about 0.45 us under full load), and what its finish leaves uncovered.  K is split where there are few tiles.
struct Cutting {
  int BN, tiles_n, chunks, splits, split_chunks;
  int64_t tiles;
  bool pair;
};
Cutting cut_product(int64_t M, int64_t N, int64_t K, int dtype, bool b_major) {
  const bool f32 = dtype != MHLA_BF16;
  Cutting best = {};
  double least = 0;
  const int chunks = static_cast<int>((K + 63) / 64);
  for (int pair = 0; pair < (f32 || M <= 128 ? 1 : 2); ++pair)
    for (int BN : {64, 128, 192, 256}) {
      if (f32 && BN > 128) break;
      if (pair && (BN == 64 || (BN == 192 && b_major))) continue;   // halves of B in whole boxes of 64
      Cutting c = {};
      c.BN = BN;
      c.pair = pair;
      c.chunks = chunks;
      c.tiles_n = static_cast<int>((N + BN - 1) / BN);
      const int64_t m = pair ? 256 : 128;
      c.tiles = (M + m - 1) / m * c.tiles_n;
      const int64_t machine = pair ? kSms / 2 : kSms;
      const double chunk_us = (f32 ? 3.0 : 1.0) * 0.45 * (128 + (pair ? BN / 2 : BN)) / 384, tail_us = 1.5 + 0.01 * BN;
      for (int splits = 1; splits <= 64; splits = splits < 8 ? splits + 1 : 2 * splits) {
        if (splits > 1 && (splits > chunks || c.tiles * (splits - 1) >= 2 * machine)) break;
        const int each = (chunks + splits - 1) / splits, used = (chunks + each - 1) / each;
        const int64_t waves = (c.tiles * used + machine - 1) / machine;
        // the parts are written and read: 8 bytes a value at 4 bytes a ns and part, and a launch
        const double us = waves * (each * chunk_us) + tail_us * (waves > 1 ? 1.3 : 1.0) +
                          (used > 1 ? 3.0 + 8e-6 * static_cast<double>(used) * M * N / 4 : 0.0);
        if (best.BN == 0 || us < least) {
          least = us;
          best = c;
          best.splits = used;
          best.split_chunks = each;
        }
      }
    }
  return best;
}
size_t part_bytes(int64_t M, int64_t N, const Cutting& c) {
  return c.splits < 2 ? 0 : align_up(static_cast<size_t>(c.splits) * M * ((N + 3) / 4 * 4) * 4);
}

template <int TERMS, bool PAIR, bool BULK = false>
int launch_product(const char* name, const Product& p, cudaStream_t s) {
  using L = GemmLay<TERMS, PAIR>;
  auto kernel = linear_gemm<TERMS, PAIR, BULK>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L::SMEM)) != cudaSuccess)
    return MHLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(L::THREADS);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  int64_t grid = 0;
  if (PAIR) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    cfg.gridDim = dim3(2);
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters < 1) return MHLA_ERR_CUDA;
    grid = 2 * std::min<int64_t>(p.units, clusters);
  } else {
    const int sms = device_sm_count();
    if (sms <= 0) return MHLA_ERR_CUDA;
    grid = std::min<int64_t>(p.units, sms);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  KernelTimer timer(name, s);
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return MHLA_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int run_product(const char* name, const Matrix& a, bool a_major, const Matrix& b, bool b_major, int64_t M, int64_t N, int64_t K,
                int dtype, const Finish& f, char* parts, cudaStream_t s) {
  const int terms = dtype == MHLA_BF16 ? 1 : 3;
  const Cutting c = cut_product(M, N, K, dtype, b_major);
  Product p = {};
  const int b_rows = c.pair ? c.BN / 2 : c.BN;
  p.a_blocks = a_major && terms == 1 && a.cols % 64 == 0;
  p.b_blocks = b_major && terms == 1 && b.cols % 64 == 0;
  if (!(p.a_blocks ? encode_blocks(&p.a, a, 2) : encode_planes(&p.a, a, terms, 64, a_major ? 64 : 128)) ||
      !(p.b_blocks ? encode_blocks(&p.b, b, b_rows / 64) : encode_planes(&p.b, b, terms, 64, b_major ? 64 : b_rows)))
    return MHLA_ERR_CUDA;
  p.f = f;
  p.parts = c.splits > 1 ? reinterpret_cast<float*>(parts) : nullptr;
  p.pitch = (N + 3) / 4 * 4;
  p.units = c.tiles * c.splits;
  p.a_major = a_major; p.b_major = b_major;
  // 32 x 32 values a warp, 64 bytes a row
  const bool bulk = c.pair && c.splits < 2 && !f.residual && N % 8 == 0;
  if (bulk) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)}, strides[1] = {static_cast<cuuint64_t>(2 * N)};
    const cuuint32_t box[2] = {32, 32};
    if (!encode_tensor_map(&p.out, 2, f.out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B) ||
        (f.pre && !encode_tensor_map(&p.pre, 2, f.pre, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B)))
      return MHLA_ERR_CUDA;
  }
  p.BN = c.BN; p.tiles_n = c.tiles_n; p.chunks = c.chunks; p.splits = c.splits; p.split_chunks = c.split_chunks;
  const int rc = terms > 1  ? launch_product<3, false>(name, p, s)
                 : bulk     ? launch_product<1, true, true>(name, p, s)
                 : c.pair   ? launch_product<1, true>(name, p, s)
                            : launch_product<1, false>(name, p, s);
  if (rc != MHLA_OK) return rc;
  if (c.splits < 2) return MHLA_OK;
  const Join j = {f, p.parts, p.pitch, c.splits};
  KernelTimer timer("linear_join", s);
  const unsigned blocks = static_cast<unsigned>((M * p.pitch / 4 + 255) / 256);
  if (terms == 1)
    linear_join<false><<<blocks, 256, 0, s>>>(j);
  else
    linear_join<true><<<blocks, 256, 0, s>>>(j);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

// Columns a thread of the planes' kernel has: 16 bytes where rows are a multiple of that.
int plane_vec(int64_t cols, int dtype) { return dtype == MHLA_BF16 ? (cols % 8 == 0 ? 8 : 1) : cols % 4 == 0 ? 4 : 1; }

int64_t plane_columns(const Planes& p, int vec) { return (p.cols + 32 * vec - 1) / (32 * vec); }

// n matrices; those that take their columns the same way in one launch.
int run_planes(const Planes* jobs, int n, int dtype, cudaStream_t s) {
  const int wide = dtype == MHLA_BF16 ? 8 : 4;
  for (int vec : {wide, 1}) {
    PlaneSet set = {};
    dim3 grid(0, 0, 0);
    for (int i = 0; i < n; ++i) {
      if (plane_vec(jobs[i].cols, dtype) != vec) continue;
      set.of[grid.z++] = jobs[i];
      grid.x = std::max(grid.x, static_cast<unsigned>(plane_columns(jobs[i], vec)));
      grid.y = std::max(grid.y, static_cast<unsigned>((jobs[i].rows + jobs[i].block_rows - 1) / jobs[i].block_rows));
    }
    if (grid.z == 0) continue;
    KernelTimer timer("linear_planes", s);
    if (dtype == MHLA_BF16) {
      if (vec > 1) linear_planes<1, 8><<<grid, 256, 0, s>>>(set);
      else linear_planes<1, 1><<<grid, 256, 0, s>>>(set);
    } else {
      if (vec > 1) linear_planes<3, 4><<<grid, 256, 0, s>>>(set);
      else linear_planes<3, 1><<<grid, 256, 0, s>>>(set);
    }
    if (cudaGetLastError() != cudaSuccess) return MHLA_ERR_CUDA;
  }
  return MHLA_OK;
}
int64_t blocks_of_rows(int64_t rows, int64_t cols, int dtype) {
  const int64_t wide = 32 * plane_vec(cols, dtype), across = (cols + wide - 1) / wide;
  int64_t n = std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, (8 * kSms + across - 1) / across));
  const int64_t each = (rows + n - 1) / n;
  return (rows + each - 1) / each;
}

// The matrix as the product reads it: as it lies, or laid out at *ws.
// A matrix as it lies, or one more of the n to be laid out.
Matrix lay_matrix(const void* x, int64_t rows, int64_t cols, int dtype, char** ws, Planes* jobs, int* n) {
  if (direct(cols, dtype)) return Matrix{x, rows, cols, cols};
  Planes& p = jobs[(*n)++];
  p = Planes{};
  p.src = x;
  p.dst = reinterpret_cast<__nv_bfloat16*>(*ws);
  p.rows = rows; p.cols = cols; p.pitch = plane_pitch(cols);
  const int64_t blocks = blocks_of_rows(rows, cols, dtype);
  p.block_rows = (rows + blocks - 1) / blocks;
  *ws += plane_bytes(rows, cols, dtype);
  return Matrix{p.dst, rows, cols, p.pitch};
}
size_t lay_bytes(int64_t rows, int64_t cols, int dtype) { return direct(cols, dtype) ? 0 : plane_bytes(rows, cols, dtype); }

// Whether linear_rows (or linear_dots) takes the call: w is read once either way, but linear_gemm is at 8 to 14 us whatever the
// rows, and linear_rows grows with rows x k.  Measured, bf16, us, linear_rows against linear_gemm for k x n: 8 rows 768 x 2304 3.2 and 9.3,
// 2304 x 768 4.3 and 8.6, 4096 x 4096 6.5 and 12.9; 16 rows 3.4 and 9.4, 5.7 and 8.6, 9.5 and 13.0; 32 rows 4.7 and 9.4, 9.1 and 8.3, 15.8 and
// 13.5; 64 rows 5.2 and 9.4, 9.2 and 8.3, 29.5 and 13.6.  linear_dots, float32, against laying out and linear_gemm, 768 x 2304 and 333 x 201: 1 row
// 7.2 and 17.2, 4.4 and 10.9; 8 rows 15.8 and 16.0, 7.5 and 10.9; 32 rows 30.3 and 16.0, 7.5 and 11.4.
constexpr int64_t kFewRows = 64, kFewProducts = 65536, kFewDots = 8;
bool few_rows(const LinearProblem& p) {
  return p.rows <= kFewDots || (direct(p.k, p.dtype) && p.rows <= kFewRows && p.rows * p.k <= kFewProducts);
}

template <int GROUPS>
int run_rows(const LinearProblem& p, const Finish& f, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.n + 15) / 16), static_cast<unsigned>((p.rows + 8 * GROUPS - 1) / (8 * GROUPS)));
  linear_rows<GROUPS><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(p.x), static_cast<const __nv_bfloat16*>(p.w), p.rows,
                                           static_cast<int32_t>(p.k), f);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

}  // namespace

size_t linear_act_workspace_bytes(const LinearProblem& p) {
  if (few_rows(p)) return 0;
  return lay_bytes(p.rows, p.k, p.dtype) + lay_bytes(p.n, p.k, p.dtype) +
         part_bytes(p.rows, p.n, cut_product(p.rows, p.n, p.k, p.dtype, false));
}

int launch_linear_act(const LinearProblem& p, const void* bias, const void* residual, void* pre, void* out, void* workspace,
                      void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Finish f = {out, pre, residual, bias, p.rows, p.n, p.act, p.n % 4 == 0};
  if (few_rows(p)) {
    KernelTimer timer("linear_rows", s);
    if (direct(p.k, p.dtype)) {
      if (p.rows <= 8) return run_rows<1>(p, f, s);
      return p.rows <= 16 ? run_rows<2>(p, f, s) : run_rows<4>(p, f, s);
    }
    const dim3 grid(static_cast<unsigned>((p.n + 7) / 8), static_cast<unsigned>((p.rows + 7) / 8));
    if (p.dtype == MHLA_BF16)
      linear_dots<__nv_bfloat16><<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(p.x), static_cast<const __nv_bfloat16*>(p.w),
                                                      p.rows, static_cast<int32_t>(p.k), f);
    else
      linear_dots<float><<<grid, 256, 0, s>>>(static_cast<const float*>(p.x), static_cast<const float*>(p.w), p.rows,
                                              static_cast<int32_t>(p.k), f);
    return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
  }
  char* ws = static_cast<char*>(workspace);
  Planes jobs[2];
  int n = 0;
  const Matrix x = lay_matrix(p.x, p.rows, p.k, p.dtype, &ws, jobs, &n), w = lay_matrix(p.w, p.n, p.k, p.dtype, &ws, jobs, &n);
  const int rc = run_planes(jobs, n, p.dtype, s);
  return rc == MHLA_OK ? run_product("linear_gemm", x, false, w, false, p.rows, p.n, p.k, p.dtype, f, ws, s) : rc;
}

size_t linear_act_bwd_workspace_bytes(const LinearProblem& p) {
  // dz (where it is not dout as it lies), x, w, the parts of either product, the sums of dz's columns
  const bool plain = p.act == MHLA_ACT_NONE && direct(p.n, p.dtype);
  const size_t parts = std::max(part_bytes(p.rows, p.k, cut_product(p.rows, p.k, p.n, p.dtype, true)),
                                part_bytes(p.n, p.k, cut_product(p.n, p.k, p.rows, p.dtype, true)));
  return (plain ? 0 : plane_bytes(p.rows, p.n, p.dtype)) + lay_bytes(p.rows, p.k, p.dtype) + lay_bytes(p.n, p.k, p.dtype) + parts +
         align_up(static_cast<size_t>(blocks_of_rows(p.rows, p.n, p.dtype) * p.n) * 4);
}

int launch_linear_act_backward(const LinearProblem& p, const void* dout, const void* pre, void* dx, void* dw, void* dbias,
                               void* workspace, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = p.dtype != MHLA_BF16, plain = p.act == MHLA_ACT_NONE && direct(p.n, p.dtype);
  char* ws = static_cast<char*>(workspace);
  Matrix dz = {dout, p.rows, p.n, p.n}, x = {}, w = {};
  Planes jobs[3];
  int n = 0;
  const int64_t blocks = blocks_of_rows(p.rows, p.n, p.dtype);
  float* sums = reinterpret_cast<float*>(ws);
  ws += align_up(static_cast<size_t>(blocks * p.n) * 4);
  if (!plain || dbias) {
    Planes& z = jobs[n++];
    z = Planes{};
    z.src = dout;
    z.pre = p.act == MHLA_ACT_NONE ? nullptr : pre;
    z.act = p.act;
    z.rows = p.rows; z.cols = p.n; z.pitch = plane_pitch(p.n);
    z.sums = dbias ? sums : nullptr;
    if (!plain) {
      z.dst = reinterpret_cast<__nv_bfloat16*>(ws);
      dz = Matrix{ws, p.rows, p.n, z.pitch};
      ws += plane_bytes(p.rows, p.n, p.dtype);
    }
    z.block_rows = (p.rows + blocks - 1) / blocks;
  }
  if (dw) x = lay_matrix(p.x, p.rows, p.k, p.dtype, &ws, jobs, &n);
  if (dx) w = lay_matrix(p.w, p.n, p.k, p.dtype, &ws, jobs, &n);
  int rc = run_planes(jobs, n, p.dtype, s);
  if (rc == MHLA_OK && dbias) {
    KernelTimer timer("linear_column_sums", s);
    const unsigned grid = static_cast<unsigned>((p.n + 7) / 8);
    if (f32)
      linear_column_sums<true><<<grid, 256, 0, s>>>(sums, dbias, p.n, static_cast<int32_t>(blocks));
    else
      linear_column_sums<false><<<grid, 256, 0, s>>>(sums, dbias, p.n, static_cast<int32_t>(blocks));
    if (cudaGetLastError() != cudaSuccess) rc = MHLA_ERR_CUDA;
  }
  Finish f = {};
  f.act = MHLA_ACT_NONE;
  f.quads = p.k % 4 == 0;
  f.N = p.k;
  if (rc == MHLA_OK && dx) {
    f.out = dx;
    f.M = p.rows;
    rc = run_product("linear_gemm_dx", dz, false, w, true, p.rows, p.k, p.n, p.dtype, f, ws, s);
  }
  if (rc == MHLA_OK && dw) {
    f.out = dw;
    f.M = p.n;
    rc = run_product("linear_gemm_dw", dz, true, x, true, p.n, p.k, p.rows, p.dtype, f, ws, s);
  }
  return rc;
}

int read_and_clear_linear_error(void* stream, uint32_t* flags) { return read_and_clear_word(g_linear_error, stream, flags); }

MHLA_DEFINE_STALL_SETTER(set_stall_linear)

}  // namespace mhla
