// Root-mean-square norm of every query and key head with the position rotation
// in the same pass, and its gradients:
//   u = x / sqrt(mean(x^2) + eps),  y = u * weight,  z = R(position) y
//   dy = R^T dz,  dx = r (weight dy - u mean(u weight dy)),  dweight = sum dy u
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "float_pairs.cuh"
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
// A group keeps its run of kHeads heads and walks the tokens: the weight stays in registers and a
// token costs three pointer steps, the rotation's row fetched once for all its heads.  The rows
// and the rotation's come by asynchronous copies a round ahead, every lane's into shared memory of
// its own: no barrier, no registers held while they are on their way.  Arithmetic works on pairs of
// channels (mul.f32x2, fma.f32x2).  Every input byte is read once and every output byte written once,
// so HBM bounds it; measured, bf16 [4, 65536, 6 + 6, 64]: forward 140 us (5.9 TB/s), gradients 207 us
// (6.0 TB/s), where one channel an instruction took 238 and loads without copies ahead 275; float32
// gradients [4, 16384, 8 + 2, 128] 158 us (6.4 TB/s).

// Four channels as they lie in memory.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using Raw = float4;
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
};

// A lane's eight channels in register pairs: the first channels of its four pairs in a, the second in b.
struct Eight {
  Two a[2], b[2];
};
__device__ __forceinline__ float low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
template <bool INTER>
__device__ __forceinline__ Eight expand(const uint2& x, const uint2& y) {
  if (INTER)
    return Eight{{two(low(x.x), low(x.y)), two(low(y.x), low(y.y))}, {two(high(x.x), high(x.y)), two(high(y.x), high(y.y))}};
  return Eight{{two(low(x.x), high(x.x)), two(low(x.y), high(x.y))}, {two(low(y.x), high(y.x)), two(low(y.y), high(y.y))}};
}
template <bool INTER>
__device__ __forceinline__ Eight expand(const float4& x, const float4& y) {
  if (INTER) return Eight{{two(x.x, x.z), two(y.x, y.z)}, {two(x.y, x.w), two(y.y, y.w)}};
  return Eight{{two(x.x, x.y), two(x.z, x.w)}, {two(y.x, y.y), two(y.z, y.w)}};
}
template <bool INTER>
__device__ __forceinline__ void round_to(const Eight& v, float4& x, float4& y) {
  float a[4], b[4];
  apart(v.a[0], a[0], a[1]); apart(v.a[1], a[2], a[3]);
  apart(v.b[0], b[0], b[1]); apart(v.b[1], b[2], b[3]);
  x = INTER ? make_float4(a[0], b[0], a[1], b[1]) : make_float4(a[0], a[1], a[2], a[3]);
  y = INTER ? make_float4(a[2], b[2], a[3], b[3]) : make_float4(b[0], b[1], b[2], b[3]);
}
template <bool INTER>
__device__ __forceinline__ void round_to(const Eight& v, uint2& x, uint2& y) {
  float4 f, g;
  round_to<INTER>(v, f, g);
  const __nv_bfloat162 p[4] = {__floats2bfloat162_rn(f.x, f.y), __floats2bfloat162_rn(f.z, f.w), __floats2bfloat162_rn(g.x, g.y),
                               __floats2bfloat162_rn(g.z, g.w)};
  x = make_uint2(*reinterpret_cast<const uint32_t*>(p), *reinterpret_cast<const uint32_t*>(p + 1));
  y = make_uint2(*reinterpret_cast<const uint32_t*>(p + 2), *reinterpret_cast<const uint32_t*>(p + 3));
}

// sum of x y over a lane's channels
__device__ __forceinline__ float dot(const Eight& x, const Eight& y) {
  Two s = mul(x.a[0], y.a[0]);
  s = fma(x.a[1], y.a[1], s);
  s = fma(x.b[0], y.b[0], s);
  s = fma(x.b[1], y.b[1], s);
  float f, g;
  apart(s, f, g);
  return f + g;
}
__device__ __forceinline__ Eight times(const Eight& x, const Eight& y) {
  return Eight{{mul(x.a[0], y.a[0]), mul(x.a[1], y.a[1])}, {mul(x.b[0], y.b[0]), mul(x.b[1], y.b[1])}};
}
__device__ __forceinline__ Eight times(const Eight& x, float y) {
  const Two t = two(y, y);
  return times(x, Eight{{t, t}, {t, t}});
}
__device__ __forceinline__ Eight times_plus(const Eight& x, const Eight& y, const Eight& z) {
  return Eight{{fma(x.a[0], y.a[0], z.a[0]), fma(x.a[1], y.a[1], z.a[1])},
               {fma(x.b[0], y.b[0], z.b[0]), fma(x.b[1], y.b[1], z.b[1])}};
}

// cos, sin and -sin of a lane's four pairs
struct Angles {
  Two c[2], s[2], ns[2];
};
__device__ __forceinline__ Eight turned(const Eight& x, const Angles& t) {
  Eight y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y.a[i] = fma(t.ns[i], x.b[i], mul(x.a[i], t.c[i]));
    y.b[i] = fma(t.s[i], x.a[i], mul(x.b[i], t.c[i]));
  }
  return y;
}

// The first `turns` pairs turned, the others left as they are: 0 times what is not finite would reach the partner.
template <bool INTER>
__device__ __forceinline__ Eight turned(const Eight& x, const Angles& t, int turns) {
  if (turns == 0) return x;
  Eight y = turned(x, t);
  if (INTER && turns < 4) {   // channels apart, pairs are turned by fours
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a[2], b[2], c[2], d[2];
      apart(x.a[i], a[0], a[1]); apart(x.b[i], b[0], b[1]);
      apart(y.a[i], c[0], c[1]); apart(y.b[i], d[0], d[1]);
      y.a[i] = two(2 * i < turns ? c[0] : a[0], 2 * i + 1 < turns ? c[1] : a[1]);
      y.b[i] = two(2 * i < turns ? d[0] : b[0], 2 * i + 1 < turns ? d[1] : b[1]);
    }
  }
  return y;
}

template <int G>
__device__ __forceinline__ float group_total(float x) {
#pragma unroll
  for (int s = G / 2; s; s >>= 1) x += __shfl_xor_sync(~0u, x, s);
  return x;
}

// How a grid's groups share the work: `slots` tokens at a time, `runs` groups each.
struct Walk {
  int64_t tokens, slots, rounds;
  int64_t step_b, step_n;   // a round in sequences and tokens of one
  int32_t runs_q, runs_k;   // runs of kHeads heads
  bool wide_rows;           // 16-byte loads of the rotation's rows
};

// Heads of a group: each group pays for its token's pointers and rotation.  Measured, gradients of bf16
// [4, 65536, 6 + 6, 64]: 214 us with 2 heads, 205 with 3; more do not fit the registers of two CTAs
// an SM.  float32 [4, 16384, 8 + 2, 128]: 171 us with 2, 155 with 1.
template <typename T>
__host__ __device__ constexpr int heads_a_group(bool bwd) {
  return sizeof(T) == 2 ? 3 : bwd ? 1 : 2;
}

// A round of a lane's rows and of its four pairs of the rotation in shared memory, every lane's
// value of one kind beside the others'.
template <typename T, bool BWD>
struct Ring {
  using R = typename Four<T>::Raw;
  static constexpr int kStages = 2, kPlanes = BWD ? 4 : 2;   // halves of x and z
  static constexpr int kRows = kPlanes * heads_a_group<T>(BWD) * 256 * static_cast<int>(sizeof(R));
  static constexpr int kStage = kRows + 2 * 256 * 16;
  static constexpr int kBytes = kStages * kStage;
  static_assert(kStages == 2, "one round is copied ahead");
};

template <typename R>
__device__ __forceinline__ void copy_ahead(R* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from), "n"(sizeof(R))
               : "memory");
}

// Where one operand's rows of a group lie, token after token.
template <typename T>
struct Rows {
  T* at;
  int64_t head, step, wrap;   // from head to head; a round; at the end of a sequence
  __device__ __forceinline__ Rows(const Operand& q, const Operand& k, bool is_k, int64_t b, int64_t n, int h0,
                                  const Walk& w, int64_t N) {
    const Operand& o = is_k ? k : q;
    head = o.sh;
    step = w.step_b * o.sb + w.step_n * o.sn;
    wrap = o.sb - N * o.sn;
    at = static_cast<T*>(o.data) + b * o.sb + n * o.sn + h0 * o.sh;
  }
  __device__ __forceinline__ void next(bool over) { at += step + (over ? wrap : 0); }
};

template <typename T, int G, bool BWD, bool INTER>
__global__ void __launch_bounds__(256, BWD ? 2 : 3) qk_norm_lanes(const QkNormProblem p, const Walk walk, float* part) {
  using R = typename Four<T>::Raw;
  constexpr int kHeads = heads_a_group<T>(BWD), kGroups = 256 / G;
  const int unit = threadIdx.x % G;
  const bool live = unit * 8 < p.d;
  // the lane's runs of channels; the four pairs 4 unit .. 4 unit + 3
  const bool pairs_here = !INTER && 4 * unit < p.pairs;
  const int c0 = pairs_here ? 4 * unit : 8 * unit, c1 = pairs_here ? 4 * unit + p.pairs : 8 * unit + 4;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const uint32_t runs = walk.runs_q + walk.runs_k;
  const uint32_t group = blockIdx.x * kGroups + threadIdx.x / G;
  const int run = static_cast<int>(group % runs);
  int64_t token = group / runs;
  const int64_t b = token / p.N;
  int64_t n = token - b * p.N;
  const bool is_k = run >= walk.runs_q;
  const int h0 = (is_k ? run - walk.runs_q : run) * kHeads;
  const int heads = live && token < walk.slots ? min(kHeads, static_cast<int>(is_k ? p.Hk : p.Hq) - h0) : 0;
  Rows<T> x(p.q, p.k, is_k, b, n, h0, walk, p.N), out(p.q_out, p.k_out, is_k, b, n, h0, walk, p.N);
  Rows<T> z = x;
  if (BWD) z = Rows<T>(p.dq_out, p.dk_out, is_k, b, n, h0, walk, p.N);
  // channel of the i-th first and second of the lane's pairs
  auto channel = [&](int i, int second) { return INTER ? 8 * unit + 2 * i + second : (second ? c1 : c0) + i; };
  Eight w;
  {
    const float* weight = is_k ? p.k_weight : p.q_weight;
    auto at = [&](int i, int second) { return weight && live ? weight[channel(i, second)] : 1.0f; };
    w = Eight{{two(at(0, 0), at(1, 0)), two(at(2, 0), at(3, 0))}, {two(at(0, 1), at(1, 1)), two(at(2, 1), at(3, 1))}};
  }
  Eight acc = {};   // the heads' share of the weight's gradient
  using Held = Ring<T, BWD>;
  extern __shared__ __align__(16) char shared[];
  int64_t token_ahead = token, n_ahead = n;
  int64_t position = 0;   // of the next round to be copied
  int turns_ahead = 0;    // pairs of the lane that the last round copied turns
  auto look_up = [&]() {
    position = n_ahead;
    if (p.positions && token_ahead < walk.tokens) position = p.positions[token_ahead];
  };
  auto copy_round = [&](int64_t round) {   // x, z and the rotation of a round, and a round on
    char* const stage = shared + static_cast<int>(round % Held::kStages) * Held::kStage;
    R* const to = reinterpret_cast<R*>(stage) + threadIdx.x;
    const int there = token_ahead < walk.tokens ? heads : 0;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (j < there) {   // what is not copied is not used, but finds zeros or an earlier round
        const T* fx = x.at + j * x.head;
        copy_ahead(to + (Held::kPlanes * j) * 256, fx + c0);
        copy_ahead(to + (Held::kPlanes * j + 1) * 256, fx + c1);
        if (BWD) {
          const T* fz = z.at + j * z.head;
          copy_ahead(to + (Held::kPlanes * j + 2) * 256, fz + c0);
          copy_ahead(to + (Held::kPlanes * j + 3) * 256, fz + c1);
        }
      }
    }
    turns_ahead = p.table && position >= 0 ? max(0, min(4, p.pairs - 4 * unit)) : 0;
    if (turns_ahead > 0 && there > 0) {
      float4* const turns = reinterpret_cast<float4*>(stage + Held::kRows) + threadIdx.x;
      const bool turned = position < p.rows;
      const float* from = p.table + 2 * (position * p.pairs + 4 * unit);
      if (turned && walk.wide_rows) {
        copy_ahead(turns, from);
        copy_ahead(turns + 256, from + 4);
      } else {
        const float past = position >= p.rows ? __int_as_float(0x7FC00000) : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2* const to = reinterpret_cast<float2*>(turns + (e >> 1) * 256) + (e & 1);
          const bool pair = 4 * unit + e < p.pairs;
          if (turned && pair)
            copy_ahead(to, from + 2 * e);
          else
            *to = make_float2(pair ? past : 1.0f, 0.0f);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    token_ahead += walk.slots;
    n_ahead += walk.step_n;
    const bool over = n_ahead >= p.N;
    if (over) n_ahead -= p.N;
    x.next(over);
    if (BWD) z.next(over);
    look_up();
  };
  if (!live)   // lanes behind the head's channels add nothing to its sums
    for (int i = 0; i < Held::kStages * Held::kPlanes * kHeads; ++i) {
      char* const stage = shared + i / (Held::kPlanes * kHeads) * Held::kStage;
      reinterpret_cast<R*>(stage)[i % (Held::kPlanes * kHeads) * 256 + threadIdx.x] = R{};
    }
  look_up();
  for (int i = 0; i < Held::kStages - 1; ++i) copy_round(i);
  // every lane of a warp takes the same number of rounds: the sums need all of them
  for (int64_t round = 0; round < walk.rounds; ++round) {
    const int count = token < walk.tokens ? heads : 0, turns = turns_ahead;
    copy_round(round + Held::kStages - 1);
    const char* const stage = shared + static_cast<int>(round % Held::kStages) * Held::kStage;
    asm volatile("cp.async.wait_group %0;" ::"n"(Held::kStages - 1) : "memory");
    float c[4] = {1.0f, 1.0f, 1.0f, 1.0f}, s[4] = {};
    if (turns > 0) {   // else none were copied
      const float4* const from = reinterpret_cast<const float4*>(stage + Held::kRows) + threadIdx.x;
      const float4 f = from[0], g = from[256];
      c[0] = f.x; s[0] = f.y; c[1] = f.z; s[1] = f.w;
      c[2] = g.x; s[2] = g.y; c[3] = g.z; s[3] = g.w;
      if (BWD)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = -s[e];
    }
    const Angles angles = {{two(c[0], c[1]), two(c[2], c[3])}, {two(s[0], s[1]), two(s[2], s[3])},
                           {two(-s[0], -s[1]), two(-s[2], -s[3])}};
    const R* const mine = reinterpret_cast<const R*>(stage) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const bool real = j < count;
      const R* const row = mine + Held::kPlanes * j * 256;
      Eight u = expand<INTER>(row[0], row[256]), y;
      const float r = rsqrtf(group_total<G>(dot(u, u)) * inv_d + p.eps);
      u = times(u, r);
      if (!BWD) {
        y = turned<INTER>(times(u, w), angles, turns);
      } else {
        y = turned<INTER>(expand<INTER>(row[2 * 256], row[3 * 256]), angles, turns);
        if (real) acc = times_plus(y, u, acc);   // eps 0: a row that is not there is 0 / 0
        y = times(y, w);
        const float m = group_total<G>(dot(y, u)) * inv_d;
        const Two down = two(-m, -m);
        y = times(times_plus(u, Eight{{down, down}, {down, down}}, y), r);
      }
      if (real) {
        R lo, hi;
        round_to<INTER>(y, lo, hi);
        *reinterpret_cast<R*>(out.at + j * out.head + c0) = lo;
        *reinterpret_cast<R*>(out.at + j * out.head + c1) = hi;
      }
    }
    token += walk.slots;
    n += walk.step_n;
    const bool over = n >= p.N;
    if (over) n -= p.N;
    out.next(over);
  }
  if (BWD) {   // the block's sums, its groups in a fixed order
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* const sums = reinterpret_cast<float*>(shared);   // in the ring's place
    static_assert(Held::kBytes >= kGroups * G * 8 * 4, "the sums fit the ring");
    __shared__ bool of_k[kGroups];
    float* mine = sums + (threadIdx.x / G) * G * 8;
    if (live)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        apart(acc.a[i], mine[channel(2 * i, 0)], mine[channel(2 * i + 1, 0)]);
        apart(acc.b[i], mine[channel(2 * i, 1)], mine[channel(2 * i + 1, 1)]);
      }
    if (unit == 0) of_k[threadIdx.x / G] = is_k;
    __syncthreads();
    if (threadIdx.x < p.d) {
      float tq = 0.0f, tk = 0.0f;
      for (int g = 0; g < kGroups; ++g) {
        const float a = sums[g * G * 8 + threadIdx.x];
        if (of_k[g])
          tk += a;
        else
          tq += a;
      }
      float* to = part + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
      to[0] = tq;
      to[128] = tk;
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
constexpr int64_t kFwdBlocks = 456;   // three

// Blocks taken; 0 when there are more heads than groups of the grid.
template <typename T, int G, bool BWD>
unsigned launch_lanes_group(const QkNormProblem& p, float* part, cudaStream_t s) {
  constexpr int kHeads = heads_a_group<T>(BWD), kGroups = 256 / G;
  const int64_t runs_q = (p.Hq + kHeads - 1) / kHeads, runs_k = (p.Hk + kHeads - 1) / kHeads, runs = runs_q + runs_k;
  Walk w;
  w.tokens = p.B * p.N;
  const int64_t blocks = (w.tokens * runs + kGroups - 1) / kGroups;
  const int64_t grid = std::min<int64_t>(blocks, BWD ? kBwdBlocks : kFwdBlocks);
  w.slots = grid * kGroups / runs;
  if (w.slots == 0) return 0;
  w.rounds = (w.tokens + w.slots - 1) / w.slots;
  w.step_b = w.slots / p.N;
  w.step_n = w.slots % p.N;
  w.runs_q = static_cast<int32_t>(runs_q);
  w.runs_k = static_cast<int32_t>(runs_k);
  w.wide_rows = p.pairs % 4 == 0 && reinterpret_cast<uintptr_t>(p.table) % 16 == 0;
  constexpr int kBytes = Ring<T, BWD>::kBytes;
  auto kernel = p.interleaved ? qk_norm_lanes<T, G, BWD, true> : qk_norm_lanes<T, G, BWD, false>;
  // a per-device setting: made on every call, for whichever device is current
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  kernel<<<static_cast<unsigned>(grid), 256, kBytes, s>>>(p, w, part);
  return static_cast<unsigned>(grid);
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
  if (in_lanes(p, false) && launch_lanes<false>(p, nullptr, s) > 0) {
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
    const bool any = p.B > 0 && p.Hq + p.Hk > 0;   // the walk over lanes needs a row
    const unsigned taken = any && in_lanes(p, true) ? launch_lanes<true>(p, part, s) : 0;
    if (taken > 0)
      grid = taken;
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
