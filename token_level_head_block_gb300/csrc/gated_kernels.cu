// Gated causal linear attention:
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
// and its gradients.  With dS_t = scale q_t do_t^T + exp(g_{t+1}) dS_{t+1},
//   dq_t = scale S_t do_t         the recurrence itself with (do, v, k) for (q, k, v)
//   dv_t = dS_t^T k_t             the recurrence run backwards with (k, q, do)
//   dk_t = dS_t v_t               the same with (v, do, q)
//   dg_t = exp(g_t) <S_{t-1}, dS_t>   a sum over pairs of tokens (gated_gate_grad below)
//
// gated_scan takes every type, size and alignment; bf16 with d <= 64 and enough tokens goes to
// the tcgen05 kernels of gated_tc_kernels.cu (wants_tc below).  A CTA walks a span of
// chunks of 64 tokens with the state (d x up to 64 columns of it) in registers.  With
// b_i the sum of the log decays of a chunk's tokens up to i and B that of all,
//   o_i = scale (e^{b_i} S^T q_i + sum_{j <= i} e^{b_i - b_j} (q_i . k_j) v_j)
//   S  <- e^B S + sum_j e^{B - b_j} k_j v_j^T
// and backwards the same with b_i the sum of the gates behind token i.
// All four products run on mma.sync m16n8k16 with float32 accumulators; what is
// not exact in bf16 enters as a sum of bf16 terms (Terms below).  When there are
// fewer (b, h) than the machine has room for, the sequence is cut into spans:
// gated_span_state forms each span's own contribution to the state,
// gated_join carries the state from span to span, and gated_scan then runs all
// spans at once.
//
// A chunk is a chain (scores, outputs, state, its planes) that few warps walk, so latency bounds it:
// measured on float32 [3, 5181, 4, 64], the tensor pipe is active 25% of the scan's time and a scheduler issues in
// one cycle of four.
// Times, all launches of a call:
//   bf16  [8, 2048, 16, 128]  forward  277 us      [4, 4096, 16, 80]  gradients 1105 us
//   f32   [8, 2048, 16, 128]  forward  816 us      [8, 6871, 4, 64]   gradients  937 us
//   f32   [3, 5181, 4, 64]    forward   86 us      [8, 4096, 16, 32]  forward    245 us
// (gated_gate_grad has 93 and 112 us of the two gradients, and the scans write 210 and 113 MB of states for it.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "gated_common.cuh"
#include "mhla_internal.h"
#include "ptx.cuh"

namespace mhla {

using namespace gated;

namespace {

constexpr int kChunk = 64;

// bf16 terms an operand enters the tensor cores with.  bf16 inputs are exact in one.
// The scores and the state a query reads feed a result that is rounded to bf16
// (2^-8) anyway: two terms leave 2^-16 there; what a token adds to the float32 state takes
// three (2^-24).  float32 runs take three everywhere.
template <typename T>
struct Terms;
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int kIn = 1, kScore = 2, kState = 2;
};
template <>
struct Terms<float> {
  static constexpr int kIn = 3, kScore = 3, kState = 3;
};
constexpr int kAdd = 3;

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Accumulators of NT column tiles.  The tensor core truncates what it adds to an
// accumulator, which drifts over a long chain: float32 runs keep the products of the
// first terms, few additions, apart from the many small ones.
template <int NT, bool APART>
struct Accumulators {
  float main[NT][4];
  float small[APART ? NT : 1][4];
  __device__ __forceinline__ float get(int n, int e) const {
    return APART ? main[n][e] + small[APART ? n : 0][e] : main[n][e];
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        main[n][e] = 0.0f;
        if (APART) small[APART ? n : 0][e] = 0.0f;
      }
  }
};

// acc[n0 .. n0 + 2 P) += A B over the terms of both whose product is not below the last
// term's size; b[t][p] holds two column tiles.  Independent accumulators follow one another.
// first: nothing is there yet.
template <int NA, int NB, int P, int NT, bool APART>
__device__ __forceinline__ void mma_terms(Accumulators<NT, APART>& acc, int n0, const uint32_t (&a)[NA][4],
                                          const uint32_t (&b)[NB][P][4], bool first = false) {
  constexpr int kMost = NA > NB ? NA : NB;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j) {
      if (i + j >= kMost) continue;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int n = n0 + 2 * p + f;
          float(&c)[4] = APART && i + j > 0 ? acc.small[APART ? n : 0] : acc.main[n];
          // the first pair of terms that goes to this accumulator
          const bool opens = APART ? (i + j == 0 || (i == NA - 1 && j == kMost - NA)) : (i == NA - 1 && j == kMost - NA);
          if (first && opens)
            mma_first(c, a[i], b[j][p][2 * f], b[j][p][2 * f + 1]);
          else
            mma(c, a[i], b[j][p][2 * f], b[j][p][2 * f + 1]);
        }
    }
}

// What a chunk needs of its gates.  Rows i of a block of 16 tokens see tokens j of other
// blocks through e^{b_i - b_j} = e^{b_i - m} e^{m - b_j}, m at the edge of the
// row's block towards them, so neither factor exceeds 1; the state, too, is read with
// e^{b_i - m} e^m.  Backwards b_i is the sum of the gates behind token i, from the chunk's end, so that what a row
// sees holds those gates alone (one that is NaN reaches no later token); all else is the same.  Within a block
// the difference of the two sums is taken itself.
struct Gates {
  float hi[kChunk], lo[kChunk];   // b_i
  float row[kChunk];              // e^{b_i - m}
  float col[4][kChunk];           // out_scale e^{m - b_j}, per block of rows
  float addw[kChunk];             // k_scale e^{B - b_j}: to the state
  float enter[4];                 // state_scale e^m
  float total;                    // e^B: of the state over the chunk
  float pad[3];
};

// A lane's two gates of a chunk (tokens 2 lane, 2 lane + 1); 0 behind the end.
template <typename T>
__device__ __forceinline__ float2 load_gates(const ScanSet& p, int64_t b, int64_t h, int64_t chunk, int lane) {
  const int64_t t = chunk * kChunk + 2 * lane;
  const T* g = static_cast<const T*>(p.g.data) + b * p.g.sb + h * p.g.sh;
  return make_float2(t < p.N ? to_f(g[t * p.g.sn]) : 0.0f, t + 1 < p.N ? to_f(g[(t + 1) * p.g.sn]) : 0.0f);
}

// One warp: the running sums and the weights of a chunk; sums: where the former go too, or null.  Returns B.
__device__ __forceinline__ Sum chunk_gates(float2 g, Gates& out, const Scan& a, int lane, float* sums = nullptr) {
  const Sum none = {0.0f, 0.0f}, first = gate_sum(g.x), second = gate_sum(g.y);
  const bool reverse = a.reverse;
  Sum run = add(first, second);
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    Sum o;
    o.hi = reverse ? __shfl_down_sync(~0u, run.hi, s) : __shfl_up_sync(~0u, run.hi, s);
    o.lo = reverse ? __shfl_down_sync(~0u, run.lo, s) : __shfl_up_sync(~0u, run.lo, s);
    if (reverse ? lane + s < 32 : lane >= s) run = add(o, run);
  }
  auto of_lane = [&](int l) {
    Sum r;
    r.hi = __shfl_sync(~0u, run.hi, l);
    r.lo = __shfl_sync(~0u, run.lo, l);
    return r;
  };
  const Sum all = of_lane(reverse ? 0 : 31);
  // at the edge of each block of rows towards what it sees
  Sum edge[4] = {of_lane(reverse ? 8 : 0), of_lane(reverse ? 16 : 7), of_lane(reverse ? 24 : 15), of_lane(23)};
  edge[reverse ? 3 : 0] = none;
  Sum next;   // of the lanes in front (behind)
  next.hi = reverse ? __shfl_down_sync(~0u, run.hi, 1) : __shfl_up_sync(~0u, run.hi, 1);
  next.lo = reverse ? __shfl_down_sync(~0u, run.lo, 1) : __shfl_up_sync(~0u, run.lo, 1);
  if (lane == (reverse ? 31 : 0)) next = none;
  const Sum at[2] = {reverse ? add(next, second) : add(next, first), reverse ? next : run};
  const int block = lane >> 3;
  Sum m = edge[0];
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (block == i) m = edge[i];
  const float2 hi = make_float2(at[0].hi, at[1].hi), lo = make_float2(at[0].lo, at[1].lo);
  const float2 row = make_float2(exp2_of(at[0], m), exp2_of(at[1], m));
  float2 addw = make_float2(exp2_of(all, at[0]), exp2_of(all, at[1]));
  addw.x *= a.k_scale;
  addw.y *= a.k_scale;
  *reinterpret_cast<float2*>(out.hi + 2 * lane) = hi;
  *reinterpret_cast<float2*>(out.lo + 2 * lane) = lo;
  if (sums) {
    *reinterpret_cast<float2*>(sums + 2 * lane) = hi;
    *reinterpret_cast<float2*>(sums + kChunk + 2 * lane) = lo;
  }
  *reinterpret_cast<float2*>(out.row + 2 * lane) = row;
  *reinterpret_cast<float2*>(out.addw + 2 * lane) = addw;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (reverse ? block <= r : block >= r) continue;   // tokens the rows of block r do not see through m
    float2 c = make_float2(exp2_of(edge[r], at[0]), exp2_of(edge[r], at[1]));
    c.x *= a.out_scale;
    c.y *= a.out_scale;
    *reinterpret_cast<float2*>(out.col[r] + 2 * lane) = c;
  }
  if ((lane & 7) == 0) out.enter[block] = a.state_scale * exp2_of(m, none);
  if (lane == 0) out.total = exp2_of(all, none);
  return all;
}

// Byte offset of a 16-byte unit of a row-major bf16 tile W columns wide.  Units change
// places with the row's number, so that eight rows read at one column (ldmatrix) or
// written at one (accumulators) meet all banks.
template <int W>
__device__ __forceinline__ int unit_at(int row, int unit) {
  return row * (2 * W) + ((unit ^ (W == 32 ? (row >> 1) & 3 : row & 7)) << 4);
}

// Warps of a CTA.  d > 64 takes eight, two to 16 rows of outputs, each with half of the columns (scores
// twice): an SM holds one or two such CTAs, too few with four warps.  [8, 2048, 16, 128] forward, four
// against eight: bf16 325, 282 us; float32 974, 816.
template <int DK>
constexpr int kWarpsOf = DK > 64 ? 8 : 4;

template <typename T, int DK, bool ASYNC>
struct Tile {
  static constexpr int kWarps = kWarpsOf<DK>, kThreads = 32 * kWarps;
  static constexpr int DV = DK < 64 ? DK : 64;     // columns of the state a CTA holds
  static constexpr int kIn = Terms<T>::kIn;
  static constexpr int kStages = ASYNC ? 2 : 1;
  static constexpr int kK = kChunk * DK * 2, kV = kChunk * DV * 2;   // bytes of a plane
  static constexpr int kS = DK * DV * 2;
  // Steps of 16 tokens or channels one after the other in a loop, where their unrolled code does not
  // stay in the instruction cache (float32, six products each): scans of [8, 6871, 4, 64] gradients 835 us
  // unrolled, 690 rolled; bf16 [8, 2048, 16, 128] 282, 293.
  static constexpr bool kRolled = Terms<T>::kIn > 1;
  // warps over the state's rows (16 each) and, for 32 rows, two halves of its columns
  static constexpr int kRowTiles = DK >= 64 ? DK / kWarps / 16 : 1;
  static constexpr int kColTiles = DK >= 64 ? DV / 8 : DV / 16;   // of eight columns
  static constexpr int kOutTiles = DV / 8 / (kWarps / 4);         // of a warp's outputs
};

// Copies chunks of one operand (columns [c0, c0 + W)) into kIn planes.
template <typename T, int W, int THREADS, bool ASYNC>
struct RowLoader {
  const T* src;
  int64_t step;      // elements: ASYNC from pass to pass, else from token to token
  int32_t width;     // columns in the tensor
  bool quads;        // float32 rows that 16-byte loads take
  __device__ __forceinline__ RowLoader(const Operand& o, int64_t b, int64_t h, int c0, int d) {
    src = static_cast<const T*>(o.data) + b * o.sb + h * o.sh + c0;
    width = min(W, d - c0);
    if constexpr (ASYNC) {
      constexpr int kUnits = W / 8, kRows = THREADS / kUnits;   // 16-byte units, rows a pass
      src += static_cast<int>(threadIdx.x) / kUnits * o.sn + 8 * (threadIdx.x % kUnits);
      step = kRows * o.sn;
    } else {
      step = o.sn;
    }
    quads = sizeof(T) == 4 && reinterpret_cast<uintptr_t>(src) % 16 == 0 && o.sn % 4 == 0 && width % 4 == 0;
  }

  // float32 rows in 16-byte units: eight of a thread in flight, `part` says which of the tile's.
  static constexpr int quads_a_part() { return kChunk * W / 4 / THREADS < 8 ? kChunk * W / 4 / THREADS : 8; }
  static constexpr int parts() { return kChunk * W / 4 / THREADS / quads_a_part(); }
  __device__ __forceinline__ void fetch(float4 (&x)[8], int part, int64_t chunk, int64_t N) const {
    const int rows = static_cast<int>(min(N - chunk * kChunk, static_cast<int64_t>(kChunk)));
    const float* from = reinterpret_cast<const float*>(src) + chunk * kChunk * step;
    constexpr int kQuads = quads_a_part();
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int i = threadIdx.x + THREADS * (part * kQuads + j), r = i / (W / 4), c = 4 * (i % (W / 4));
      x[j] = r < rows && c < width ? *reinterpret_cast<const float4*>(from + r * step + c)
                                   : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
  __device__ __forceinline__ void put(char* dst, const float4 (&x)[8], int part) const {
    constexpr int kQuads = quads_a_part();
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int i = threadIdx.x + THREADS * (part * kQuads + j), r = i / (W / 4), c = 4 * (i % (W / 4));
      float a[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int n = 0; n < Terms<T>::kIn; ++n) {
        const uint32_t lo = pack(a[0], a[1]), hi = pack(a[2], a[3]);
        *reinterpret_cast<uint2*>(dst + n * kChunk * W * 2 + unit_at<W>(r, c >> 3) + (c & 7) * 2) = make_uint2(lo, hi);
        const float f[4] = {low(lo), high(lo), low(hi), high(hi)};
        // an infinity is its first term alone
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = fabsf(f[e]) < __int_as_float(0x7F800000) ? a[e] - f[e] : 0.0f;
      }
    }
  }
  // Asks L2 for a later chunk's rows.
  __device__ __forceinline__ void prefetch(int64_t chunk, int64_t N) const {
    constexpr int kLine = 128 / sizeof(T), kLines = (W + kLine - 1) / kLine;
    const int rows = static_cast<int>(min(N - chunk * kChunk, static_cast<int64_t>(kChunk)));
#pragma unroll
    for (int i0 = 0; i0 < kChunk * kLines; i0 += THREADS) {
      const int i = i0 + threadIdx.x, r = i / kLines, c = kLine * (i % kLines);
      if (r < rows && c < width)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + (chunk * kChunk + r) * step + c));
    }
  }
  __device__ __forceinline__ void load(char* dst, int64_t chunk, int64_t N) const {
    const int rows = static_cast<int>(min(N - chunk * kChunk, static_cast<int64_t>(kChunk)));
    if constexpr (ASYNC) {
      constexpr int kUnits = W / 8, kRows = THREADS / kUnits, kSteps = kChunk / kRows;
      const int r = threadIdx.x / kUnits, u = threadIdx.x % kUnits;
      if (8 * u >= width) return;   // the columns behind d were zeroed at the start
      static_assert(kRows % 8 == 0, "a pass keeps the units' places");
      const uint32_t at = ptx::smem_u32(dst) + unit_at<W>(r, u);
      const T* x = src + chunk * (kSteps * step);
      if (rows == kChunk) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i, x += step) cp_async_16(at + i * kRows * W * 2, x, 16);
      } else {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const bool in = r + i * kRows < rows;
          cp_async_16(at + i * kRows * W * 2, in ? x + i * step : static_cast<const T*>(src), in ? 16 : 0);
        }
      }
    } else {
      constexpr int kPairs = kChunk * W / 2 / THREADS, kBatch = kPairs < 8 ? kPairs : 8;   // loads in flight
      for (int i0 = 0; i0 < kPairs; i0 += kBatch) {
        float a[kBatch], e[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int i = threadIdx.x + THREADS * (i0 + j), r = i / (W / 2), c = 2 * (i % (W / 2));
          const T* x = src + (chunk * kChunk + r) * step + c;
          a[j] = r < rows && c < width ? to_f(x[0]) : 0.0f;
          e[j] = r < rows && c + 1 < width ? to_f(x[1]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int i = threadIdx.x + THREADS * (i0 + j), r = i / (W / 2), c = 2 * (i % (W / 2));
#pragma unroll
          for (int n = 0; n < Terms<T>::kIn; ++n) {
            const uint32_t p = pack(a[j], e[j]);
            *reinterpret_cast<uint32_t*>(dst + n * kChunk * W * 2 + unit_at<W>(r, c >> 3) + (c & 7) * 2) = p;
            // an infinity is its first term alone
            a[j] = fabsf(low(p)) < __int_as_float(0x7F800000) ? a[j] - low(p) : 0.0f;
            e[j] = fabsf(high(p)) < __int_as_float(0x7F800000) ? e[j] - high(p) : 0.0f;
          }
        }
      }
    }
  }
};

// One operand's chunk after the other, float32 rows in 16-byte units where all allow it: the next
// part's loads are in flight while one is split into its terms.
template <typename T, int W, int THREADS>
struct PlainPart {
  const RowLoader<T, W, THREADS, false>& rows;
  char* dst;
};
template <typename... P>
__device__ __forceinline__ void fetch_first(float4 (&x)[8], int64_t chunk, int64_t N, const P&... parts) {
  if constexpr (sizeof...(P) > 0) {
    auto first = [&](const auto& p, const auto&...) { p.rows.fetch(x, 0, chunk, N); };
    first(parts...);
  }
}
template <typename T, int THREADS, int W0, int... W>
__device__ __forceinline__ void load_plain(int64_t chunk, int64_t N, PlainPart<T, W0, THREADS> one,
                                           PlainPart<T, W, THREADS>... more) {
  if constexpr (sizeof(T) == 4) {
    if ((one.rows.quads && ... && more.rows.quads)) {
      float4 x[2][8];
      int turn = 0;
      one.rows.fetch(x[0], 0, chunk, N);
      auto rest = [&](auto& self, const auto& now, const auto&... next) -> void {
        using Rows = std::remove_reference_t<decltype(now.rows)>;
#pragma unroll
        for (int part = 0; part < Rows::parts(); ++part) {
          if (part + 1 < Rows::parts())
            now.rows.fetch(x[turn ^ 1], part + 1, chunk, N);
          else
            fetch_first(x[turn ^ 1], chunk, N, next...);
          now.rows.put(now.dst, x[turn], part);
          turn ^= 1;
        }
        if constexpr (sizeof...(next) > 0) self(self, next...);
      };
      rest(rest, one, more...);
      return;
    }
  }
  one.rows.load(one.dst, chunk, N);
  (more.rows.load(more.dst, chunk, N), ...);
}

// A state as gated_scan's threads hold it: for each tile of eight columns that the state meets, 16 bytes of every thread
// whose rows it meets.
struct Held {
  int threads, quads;   // a tile's, a state's
};
template <int DK>
__host__ __device__ constexpr Held held_state(int d) {
  const int threads = DK > 32 ? 32 * ((d + 15) / 16) : 128;
  return Held{threads, threads * (DK > 32 ? (d + 7) / 8 : 2)};
}

// Each thread's part of the state: row tile m, column tile n, the four values of
// an mma accumulator.  `row` and `col` are those of the first.
template <int DK>
struct StatePlace {
  int row, col;
  __device__ __forceinline__ StatePlace(int warp, int lane) {
    row = (DK >= 64 ? DK / kWarpsOf<DK> * warp : 16 * (warp & 1)) + (lane >> 2);
    col = (DK >= 64 ? 0 : 16 * (warp >> 1)) + 2 * (lane & 3);
  }
};

// S <- e^B S + (addw k)^T v over one k-step of 16 tokens: the scaled, split
// transpose of k's rows for this warp's state rows.
template <typename T, int DK, bool ASYNC>
__device__ __forceinline__ void add_operand(uint32_t (&a)[kAdd][4], uint32_t k_base, int row_tile, int step,
                                            const float* addw, int lane) {
  using L = Tile<T, DK, ASYNC>;
  const int token = 16 * step + (lane & 7) + ((lane >> 4) & 1) * 8, r = row_tile + ((lane >> 3) & 1) * 8;
  const float2 w0 = *reinterpret_cast<const float2*>(addw + 16 * step + 2 * (lane & 3));
  const float2 w1 = *reinterpret_cast<const float2*>(addw + 16 * step + 8 + 2 * (lane & 3));
  float x[4][2];
#pragma unroll
  for (int n = 0; n < L::kIn; ++n) {
    uint32_t k[4];
    ldsm_t(k, k_base + n * L::kK + unit_at<DK>(token, r >> 3));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e][0] = n == 0 ? low(k[e]) : x[e][0] + low(k[e]);
      x[e][1] = n == 0 ? high(k[e]) : x[e][1] + high(k[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 w = e < 2 ? w0 : w1;
    uint32_t t[kAdd];
    split<kAdd>(x[e][0] * w.x, x[e][1] * w.y, t);
#pragma unroll
    for (int i = 0; i < kAdd; ++i) a[i][e] = t[i];
  }
}

// Fragments of 16 tokens by 16 columns of a row-major plane [token][column]
// (v, or the state with r for the token): two column tiles of B operands.
template <int W>
__device__ __forceinline__ uint32_t column_address(uint32_t base, int token0, int col0, int lane) {
  return base + unit_at<W>(token0 + (lane & 7) + ((lane >> 3) & 1) * 8, (col0 >> 3) + (lane >> 4));
}

// S <- e^B S + sum over a chunk's tokens of (addw k)^T v.  The chunk's sum is formed apart
// and added once, rounded to nearest: a long sequence must not gather the tensor
// core's truncation.
template <typename T, int DK, bool ASYNC>
__device__ __forceinline__ void add_chunk(float (&S)[Tile<T, DK, ASYNC>::kRowTiles][Tile<T, DK, ASYNC>::kColTiles][4],
                                          uint32_t k_base, uint32_t v_base, const Gates& w, int warp, int lane) {
  using L = Tile<T, DK, ASYNC>;
  constexpr int P = L::kColTiles / 2;
  const int row0 = DK >= 64 ? DK / kWarpsOf<DK> * warp : 16 * (warp & 1), col0 = DK >= 64 ? 0 : 16 * (warp >> 1);
  const float total = w.total;
#pragma unroll
  for (int m = 0; m < L::kRowTiles; ++m) {
    Accumulators<L::kColTiles, (L::kIn > 1)> sum;
    if (L::kRolled) sum.clear();
#pragma unroll(L::kRolled ? 1 : kChunk / 16)
    for (int s = 0; s < kChunk / 16; ++s) {
      uint32_t ka[kAdd][4], vb[L::kIn][P][4];
#pragma unroll
      for (int t = 0; t < L::kIn; ++t)
#pragma unroll
        for (int n = 0; n < P; ++n)
          ldsm_t(vb[t][n], column_address<L::DV>(v_base + t * L::kV, 16 * s, col0 + 16 * n, lane));
      add_operand<T, DK, ASYNC>(ka, k_base, row0 + 16 * m, s, w.addw, lane);
      mma_terms(sum, 0, ka, vb, !L::kRolled && s == 0);
    }
#pragma unroll
    for (int n = 0; n < L::kColTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[m][n][e] = fmaf(total, S[m][n][e], sum.get(n, e));
  }
}

template <typename T, int DK, bool ASYNC>
__global__ void __launch_bounds__(32 * kWarpsOf<DK>) gated_span_state(const __grid_constant__ ScanSet p) {
  using L = Tile<T, DK, ASYNC>;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) Gates gates[2];
  constexpr int kStage = L::kIn * (L::kK + L::kV);
  const Scan& a = p.scan[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the span last in order adds to no other
  const int64_t nspans = p.spans - 1;
  int64_t id = blockIdx.x;
  const int64_t span = id % nspans + (a.reverse ? 1 : 0);
  id /= nspans;
  const int slices = (p.d + L::DV - 1) / L::DV;
  const int c0 = static_cast<int>(id % slices) * L::DV;
  const int64_t bh = id / slices, b = bh / p.H, h = bh % p.H;
  const int64_t first = span * p.span_chunks;
  const int count = static_cast<int>(min(p.span_chunks, p.chunks - first));
  const bool reverse = a.reverse;

  if constexpr (ASYNC) {   // columns behind d stay zero
    for (int i = threadIdx.x; i < L::kStages * kStage / 16; i += L::kThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  const RowLoader<T, DK, L::kThreads, ASYNC> rows_k(a.k, b, h, 0, p.d);
  const RowLoader<T, L::DV, L::kThreads, ASYNC> rows_v(a.v, b, h, c0, p.d);
  auto chunk_of = [&](int i) { return first + (reverse ? count - 1 - i : i); };
  auto load = [&](int i) {
    char* st = smem + (i % L::kStages) * kStage;
    if constexpr (ASYNC) {
      rows_k.load(st, chunk_of(i), p.N);
      rows_v.load(st + L::kIn * L::kK, chunk_of(i), p.N);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      load_plain(chunk_of(i), p.N, PlainPart<T, DK, L::kThreads>{rows_k, st},
                 PlainPart<T, L::DV, L::kThreads>{rows_v, st + L::kIn * L::kK});
    }
  };

  float S[L::kRowTiles][L::kColTiles][4] = {};
  Sum all = {0.0f, 0.0f};
  float2 g = make_float2(0.0f, 0.0f);
  if (warp == 0) {
    all = chunk_gates(load_gates<T>(p, b, h, chunk_of(0), lane), gates[0], a, lane);
    if (count > 1) g = load_gates<T>(p, b, h, chunk_of(1), lane);
  }
  if constexpr (ASYNC) load(0);
  for (int i = 0; i < count; ++i) {
    if constexpr (ASYNC) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      if (i + 1 < count) load(i + 1);
    } else {
      __syncthreads();
      load(i);
      if (i + 1 < count) {
        rows_k.prefetch(chunk_of(i + 1), p.N);
        rows_v.prefetch(chunk_of(i + 1), p.N);
      }
      __syncthreads();
    }
    if (warp == 0 && i + 1 < count) {
      all = add(all, chunk_gates(g, gates[(i + 1) & 1], a, lane));
      if (i + 2 < count) g = load_gates<T>(p, b, h, chunk_of(i + 2), lane);
    }
    const uint32_t k_base = ptx::smem_u32(smem + (i % L::kStages) * kStage);
    add_chunk<T, DK, ASYNC>(S, k_base, k_base + L::kIn * L::kK, gates[i & 1], warp, lane);
  }
  const StatePlace<DK> at(warp, lane);
  float* out = a.local + (bh * p.spans + span) * p.d * p.d;
#pragma unroll
  for (int m = 0; m < L::kRowTiles; ++m)
#pragma unroll
    for (int n = 0; n < L::kColTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = at.row + 16 * m + (e >> 1) * 8, c = c0 + at.col + 8 * n + (e & 1);
        if (r < p.d && c < p.d) out[r * p.d + c] = S[m][n][e];
      }
  if (c0 == 0 && threadIdx.x == 0) a.decay[bh * p.spans + span] = exp2f(all.hi + all.lo);
}

// Turns every span's own contribution into the state that enters the span, in
// order of the scan; one thread an element of one (b, h)'s state.  The spans' values come from L2, eight loads
// in flight: 5 us for 25 spans of 12 (b, h) with d = 64, most of it the launch.
__global__ void __launch_bounds__(256) gated_join(const __grid_constant__ ScanSet p) {
  const Scan& a = p.scan[blockIdx.y];
  const int64_t dd = static_cast<int64_t>(p.d) * p.d;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.BH * dd) return;
  const int64_t bh = i / dd, e = i % dd;
  const int64_t r = e / p.d, c = e % p.d;
  float S = a.init ? a.init[bh * dd + (a.init_transposed ? c * p.d + r : e)] : 0.0f;
  const int64_t n = p.spans;
  float* at = a.local + (bh * n + (a.reverse ? n - 1 : 0)) * dd + e;
  const float* w = a.decay + bh * n + (a.reverse ? n - 1 : 0);
  const int64_t step = a.reverse ? -dd : dd, wstep = a.reverse ? -1 : 1;
  constexpr int kBatch = 8;   // loads in flight
  for (int64_t s = 0; s < n; s += kBatch) {
    float own[kBatch], f[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (s + j < n - 1) {
        own[j] = at[j * step];
        f[j] = w[j * wstep];
      }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (s + j < n) {
        at[j * step] = S;
        if (s + j < n - 1) S = fmaf(f[j], S, own[j]);
      }
    at += kBatch * step;
    w += kBatch * wstep;
  }
}

template <typename T, int DK, bool ASYNC>
struct ScanShared {
  using L = Tile<T, DK, ASYNC>;
  static constexpr int kStage = L::kIn * (2 * L::kK + L::kV);   // q, k, v
  static constexpr int kBytes = L::kStages * kStage + Terms<T>::kState * L::kS;
};

// The outputs of a chunk for one warp's 16 rows: what they read from the state,
// the tokens of other blocks, then their own block's.  of_state(o) looks at the first of these, times its row's decay.
template <typename T, int DK, bool ASYNC, bool REVERSE, typename OfState>
__device__ __forceinline__ void read_chunk(Accumulators<Tile<T, DK, ASYNC>::kOutTiles, (Terms<T>::kIn > 1)>& o,
                                           const char* stage, uint32_t s_base, const Gates& w, float out_scale, int own, int col0,
                                           int lane, OfState of_state) {
  using L = Tile<T, DK, ASYNC>;
  constexpr int kScore = Terms<T>::kScore, kState = Terms<T>::kState, NV = L::kOutTiles, P = NV / 2, kSteps = kChunk / 16;
  constexpr bool kApart = L::kIn > 1;
  const uint32_t q_base = ptx::smem_u32(stage), k_base = q_base + L::kIn * L::kK, v_base = k_base + L::kIn * L::kK;
  const int rows0 = 16 * own, row = rows0 + (lane >> 2);
  Accumulators<2 * kSteps, kApart> sc;
  if (L::kRolled) {
    o.clear();
    sc.clear();
  }
#pragma unroll(L::kRolled ? 1 : DK / 16)
  for (int ks = 0; ks < DK / 16; ++ks) {
    uint32_t qa[L::kIn][4];
#pragma unroll
    for (int t = 0; t < L::kIn; ++t)
      ldsm(qa[t], q_base + t * L::kK + unit_at<DK>(rows0 + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * ks + (lane >> 4)));
    uint32_t sb[kState][P][4];
#pragma unroll
    for (int t = 0; t < kState; ++t)
#pragma unroll
      for (int n = 0; n < P; ++n)
        ldsm_t(sb[t][n], column_address<L::DV>(s_base + t * L::kS, 16 * ks, col0 + 16 * n, lane));
    mma_terms(o, 0, qa, sb, !L::kRolled && ks == 0);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if (REVERSE ? s < own : s > own) continue;
      uint32_t kb[L::kIn][1][4];
#pragma unroll
      for (int t = 0; t < L::kIn; ++t)
        ldsm(kb[t][0],
             k_base + t * L::kK + unit_at<DK>(16 * s + (lane & 7) + (lane >> 4) * 8, 2 * ks + ((lane >> 3) & 1)));
      mma_terms(sc, 2 * s, qa, kb, !L::kRolled && ks == 0);
    }
  }
  const float enter = w.enter[own];
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o.main[n][e] = enter * o.get(n, e);
      if (kApart) o.small[kApart ? n : 0][e] = 0.0f;
    }
  of_state(o);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    if (REVERSE ? s <= own : s >= own) continue;
    uint32_t pa[kScore][4], vb[L::kIn][P][4];
#pragma unroll
    for (int t = 0; t < L::kIn; ++t)
#pragma unroll
      for (int n = 0; n < P; ++n)
        ldsm_t(vb[t][n], column_address<L::DV>(v_base + t * L::kV, 16 * s, col0 + 16 * n, lane));
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const float2 c = *reinterpret_cast<const float2*>(w.col[own] + 16 * s + 8 * f + 2 * (lane & 3));
      uint32_t t0[kScore], t1[kScore];
      split<kScore>(sc.get(2 * s + f, 0) * c.x, sc.get(2 * s + f, 1) * c.y, t0);
      split<kScore>(sc.get(2 * s + f, 2) * c.x, sc.get(2 * s + f, 3) * c.y, t1);
#pragma unroll
      for (int t = 0; t < kScore; ++t) {
        pa[t][2 * f] = t0[t];
        pa[t][2 * f + 1] = t1[t];
      }
    }
    mma_terms(o, 0, pa, vb);
  }
  const float row0 = w.row[row], row1 = w.row[row + 8];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    o.main[n][0] *= row0; o.main[n][1] *= row0;
    o.main[n][2] *= row1; o.main[n][3] *= row1;
    if (kApart) {
      float* x = o.small[kApart ? n : 0];
      x[0] *= row0; x[1] *= row0;
      x[2] *= row1; x[3] *= row1;
    }
  }
  // the own block: the scores that a row sees
  float own_sc[2][4] = {};
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    if (s == own)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) own_sc[f][e] = sc.get(2 * s + f, e);
  const float bh0 = w.hi[row], bl0 = w.lo[row], bh1 = w.hi[row + 8], bl1 = w.lo[row + 8];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    const int j = rows0 + 8 * f + 2 * (lane & 3);
    const float2 hj = *reinterpret_cast<const float2*>(w.hi + j), lj = *reinterpret_cast<const float2*>(w.lo + j);
    float x[4] = {(bh0 - hj.x) + (bl0 - lj.x), (bh0 - hj.y) + (bl0 - lj.y), (bh1 - hj.x) + (bl1 - lj.x),
                  (bh1 - hj.y) + (bl1 - lj.y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = row + (e >> 1) * 8, c = j + (e & 1);
      const bool keep = REVERSE ? c >= r : c <= r;
      own_sc[f][e] = keep ? own_sc[f][e] * (out_scale * exp2_fast(x[e])) : 0.0f;
    }
  }
  uint32_t vb[L::kIn][P][4];
#pragma unroll
  for (int t = 0; t < L::kIn; ++t)
#pragma unroll
    for (int n = 0; n < P; ++n)
      ldsm_t(vb[t][n], column_address<L::DV>(v_base + t * L::kV, rows0, col0 + 16 * n, lane));
  // A row of v that holds an infinity or NaN must not reach the rows that do not see
  // it (0 times infinity): such a block goes without the tensor core.
  uint32_t bad = 0;
#pragma unroll
  for (int n = 0; n < P; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 z = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&vb[0][n][e]),
                                       __floats2bfloat162_rn(0.0f, 0.0f));
      bad |= *reinterpret_cast<const uint32_t*>(&z);
    }
  if (!__any_sync(~0u, bad & 0x7FFF7FFFu)) {
    uint32_t pa[kScore][4];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      uint32_t t0[kScore], t1[kScore];
      split<kScore>(own_sc[f][0], own_sc[f][1], t0);
      split<kScore>(own_sc[f][2], own_sc[f][3], t1);
#pragma unroll
      for (int t = 0; t < kScore; ++t) {
        pa[t][2 * f] = t0[t];
        pa[t][2 * f + 1] = t1[t];
      }
    }
    mma_terms(o, 0, pa, vb);
  } else {
    const char* v = stage + 2 * L::kIn * L::kK;
#pragma unroll 1
    for (int j = 0; j < 16; ++j) {
      const int src = (lane & ~3) | ((j & 7) >> 1);
      float x[4];   // (row, j): column tile j / 8, value j % 2 of its lane; (row + 8, j): the two behind
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __shfl_sync(~0u, j < 8 ? own_sc[0][e] : own_sc[1][e], src);
      const float up = j & 1 ? x[1] : x[0], dn = j & 1 ? x[3] : x[2];
      const int r = lane >> 2;
      const bool sees_up = REVERSE ? j >= r : j <= r, sees_dn = REVERSE ? j >= r + 8 : j <= r + 8;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = 0.0f;
#pragma unroll
          for (int t = 0; t < L::kIn; ++t)
            y += __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(v + t * L::kV + unit_at<L::DV>(rows0 + j, col0 / 8 + n) +
                                                                          2 * (2 * (lane & 3) + e)));
          if (sees_up) o.main[n][e] = fmaf(up, y, o.main[n][e]);
          if (sees_dn) o.main[n][2 + e] = fmaf(dn, y, o.main[n][2 + e]);
        }
    }
  }
}

// GRAD: what the gates' gradient needs is written too.
template <typename T, int DK, bool ASYNC, bool GRAD>
__global__ void __launch_bounds__(32 * kWarpsOf<DK>, DK <= (sizeof(T) == 2 ? 64 : 32) ? 3 : 1)
    gated_scan(const __grid_constant__ ScanSet p) {
  using L = Tile<T, DK, ASYNC>;
  using M = ScanShared<T, DK, ASYNC>;
  constexpr int kState = Terms<T>::kState, NV = L::kOutTiles;
  extern __shared__ __align__(16) char smem[];
  __shared__ __align__(16) Gates gates[2];
  const Scan& a = p.scan[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t id = blockIdx.x;
  const int64_t span = id % p.spans;
  id /= p.spans;
  const int slices = (p.d + L::DV - 1) / L::DV;
  const int slice = static_cast<int>(id % slices), c0 = slice * L::DV;
  const int64_t bh = id / slices, b = bh / p.H, h = bh % p.H;
  const int64_t first = span * p.span_chunks;
  const int count = static_cast<int>(min(p.span_chunks, p.chunks - first));
  const bool reverse = a.reverse;
  // Rows later in the order see more of the chunk: neighbouring CTAs give them
  // to different warps, so that an SM's four schedulers get the same work.
  const int own = (warp + static_cast<int>(blockIdx.x)) & 3, rows0 = 16 * own;
  const int half = warp >> 2, col0 = 8 * NV * half;   // this warp's columns of the outputs
  char* planes = smem + L::kStages * M::kStage;
  const uint32_t s_base = ptx::smem_u32(planes);

  if constexpr (ASYNC) {
    for (int i = threadIdx.x; i < L::kStages * M::kStage / 16; i += L::kThreads)
      reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  const RowLoader<T, DK, L::kThreads, ASYNC> rows_q(a.q, b, h, 0, p.d), rows_k(a.k, b, h, 0, p.d);
  const RowLoader<T, L::DV, L::kThreads, ASYNC> rows_v(a.v, b, h, c0, p.d);
  auto chunk_of = [&](int i) { return first + (reverse ? count - 1 - i : i); };
  auto load = [&](int i) {
    char* st = smem + (i % L::kStages) * M::kStage;
    if constexpr (ASYNC) {
      rows_q.load(st, chunk_of(i), p.N);
      rows_k.load(st + L::kIn * L::kK, chunk_of(i), p.N);
      rows_v.load(st + 2 * L::kIn * L::kK, chunk_of(i), p.N);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      load_plain(chunk_of(i), p.N, PlainPart<T, DK, L::kThreads>{rows_q, st},
                 PlainPart<T, DK, L::kThreads>{rows_k, st + L::kIn * L::kK},
                 PlainPart<T, L::DV, L::kThreads>{rows_v, st + 2 * L::kIn * L::kK});
    }
  };
  if constexpr (ASYNC) load(0);

  // the state entering the span
  const StatePlace<DK> at(warp, lane);
  float S[L::kRowTiles][L::kColTiles][4];
  {
    const float* in = a.init ? a.init + (bh * a.init_spans + (a.init_spans > 1 ? span : 0)) * p.d * p.d : nullptr;
#pragma unroll
    for (int m = 0; m < L::kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < L::kColTiles; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = at.row + 16 * m + (e >> 1) * 8, c = c0 + at.col + 8 * n + (e & 1);
          S[m][n][e] = in && r < p.d && c < p.d ? in[a.init_transposed ? c * p.d + r : r * p.d + c] : 0.0f;
        }
  }
  auto publish = [&]() {   // the state as bf16 terms for the queries
#pragma unroll
    for (int m = 0; m < L::kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < L::kColTiles; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t t[kState];
          split<kState>(S[m][n][2 * e], S[m][n][2 * e + 1], t);
#pragma unroll
          for (int k = 0; k < kState; ++k)
            *reinterpret_cast<uint32_t*>(planes + k * L::kS + unit_at<L::DV>(at.row + 16 * m + 8 * e, (at.col >> 3) + n) +
                                         4 * (lane & 3)) = t[k];
        }
  };
  publish();

  // the warps take the gates of the chunks in turn, a chunk ahead
  float2 g = make_float2(0.0f, 0.0f);
  auto sums_of = [&](int i) {
    return GRAD && a.sums && slice == 0 ? a.sums + (bh * p.chunks + chunk_of(i)) * (2 * kChunk) : nullptr;
  };
  if (warp == 0) chunk_gates(load_gates<T>(p, b, h, chunk_of(0), lane), gates[0], a, lane, sums_of(0));
  if (warp == 1 && count > 1) g = load_gates<T>(p, b, h, chunk_of(1), lane);

  T* const out = static_cast<T*>(a.out.data) + b * a.out.sb + h * a.out.sh + c0;
  for (int i = 0; i < count; ++i) {
    if constexpr (ASYNC) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      if (i + 1 < count) load(i + 1);
    } else {
      __syncthreads();
      load(i);
      if (i + 1 < count) {
        rows_q.prefetch(chunk_of(i + 1), p.N);
        rows_k.prefetch(chunk_of(i + 1), p.N);
        rows_v.prefetch(chunk_of(i + 1), p.N);
      }
      __syncthreads();
    }
    if (i + 1 < count && warp == ((i + 1) & 3)) chunk_gates(g, gates[(i + 1) & 1], a, lane, sums_of(i + 1));
    if (i + 2 < count && warp == ((i + 2) & 3)) g = load_gates<T>(p, b, h, chunk_of(i + 2), lane);
    char* stage = smem + (i % L::kStages) * M::kStage;
    const Gates& w = gates[i & 1];
    const int row = rows0 + (lane >> 2);
    const int64_t t0 = chunk_of(i) * kChunk;
    {
      Accumulators<NV, (L::kIn > 1)> o;
      // a row's dot with what it reads from the state, for the gates' gradient
      auto of_state = [&](const Accumulators<NV, (L::kIn > 1)>& o) {
        if (!GRAD || !a.dots) return;
        const T* dot = static_cast<const T*>(a.dot.data) + b * a.dot.sb + h * a.dot.sh + c0;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float sum = 0.0f;
          const int64_t t = t0 + row + 8 * f;
          if (t < p.N) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              const int c = col0 + 8 * n + 2 * (lane & 3);
              const T* x = dot + t * a.dot.sn + c;
              if constexpr (ASYNC) {
                if (c0 + c < p.d) {
                  const uint32_t xx = *reinterpret_cast<const uint32_t*>(x);
                  sum = fmaf(o.main[n][2 * f], low(xx), fmaf(o.main[n][2 * f + 1], high(xx), sum));
                }
              } else {
                if (c0 + c < p.d) sum = fmaf(o.main[n][2 * f], to_f(x[0]), sum);
                if (c0 + c + 1 < p.d) sum = fmaf(o.main[n][2 * f + 1], to_f(x[1]), sum);
              }
            }
          }
          sum += __shfl_xor_sync(~0u, sum, 1);
          sum += __shfl_xor_sync(~0u, sum, 2);
          if ((lane & 3) == 0 && t < p.N)
            a.dots[((slice * (L::kWarps / 4) + half) * p.BH + bh) * p.N + t] = w.row[row + 8 * f] * sum;
        }
      };
      if (reverse)
        read_chunk<T, DK, ASYNC, true>(o, stage, s_base, w, a.out_scale, own, col0, lane, of_state);
      else
        read_chunk<T, DK, ASYNC, false>(o, stage, s_base, w, a.out_scale, own, col0, lane, of_state);

      // rows out: rounded once, through this warp's own rows of q
      if constexpr (ASYNC) {
        if (L::kWarps == 4)
          __syncwarp();   // every lane has read its rows of q
        else              // and every lane of the warp with the other columns
          asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");
        // the columns behind d stay zero (a NaN row would put NaN there)
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int f = 0; f < 2; ++f)
            if (c0 + col0 + 8 * n < p.d)
              *reinterpret_cast<uint32_t*>(stage + unit_at<DK>(row + 8 * f, col0 / 8 + n) + 4 * (lane & 3)) =
                  pack(o.get(n, 2 * f), o.get(n, 2 * f + 1));
        __syncwarp();
        constexpr int kUnits = NV;
        const int r = lane / kUnits, c = col0 + 8 * (lane % kUnits);
        const int64_t t = t0 + rows0 + r;
        T* to = out + t * a.out.sn + c;
#pragma unroll
        for (int u = 0; u < 16 * kUnits / 32; ++u) {
          constexpr int kStep = 32 / kUnits;   // rows a pass
          if (t + u * kStep < p.N && c0 + c < p.d)
            *reinterpret_cast<uint4*>(to + u * kStep * a.out.sn) =
                *reinterpret_cast<const uint4*>(stage + unit_at<DK>(rows0 + r + u * kStep, c >> 3));
        }
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int64_t t = t0 + row + 8 * f;
          if (t >= p.N) continue;
#pragma unroll
          for (int n = 0; n < NV; ++n) {
            const int c = col0 + 8 * n + 2 * (lane & 3);
            if (c0 + c < p.d) from_f(out + t * a.out.sn + c, o.get(n, 2 * f));
            if (c0 + c + 1 < p.d) from_f(out + t * a.out.sn + c + 1, o.get(n, 2 * f + 1));
          }
        }
      }
    }
    if (GRAD && a.entries) {
      static_assert(L::kRowTiles == 1, "16 rows a warp");
      const Held held = held_state<DK>(p.d);
      float4* to = reinterpret_cast<float4*>(a.entries) + (bh * p.chunks + chunk_of(i)) * held.quads +
                   slice * L::kColTiles * held.threads + threadIdx.x;
#pragma unroll
      for (int n = 0; n < L::kColTiles; ++n, to += held.threads)
        if (DK == 32 || (at.row - (lane >> 2) < p.d && c0 + 8 * n < p.d)) *to = make_float4(S[0][n][0], S[0][n][1], S[0][n][2], S[0][n][3]);
    }
    const uint32_t k_base = ptx::smem_u32(stage) + L::kIn * L::kK;
    add_chunk<T, DK, ASYNC>(S, k_base, k_base + L::kIn * L::kK, w, warp, lane);
    if (i + 1 < count) {
      __syncthreads();   // every warp has read the state's planes
      publish();
    }
  }
  if (a.last && span == (reverse ? 0 : p.spans - 1)) {
    float* last = a.last + bh * p.d * p.d;
#pragma unroll
    for (int m = 0; m < L::kRowTiles; ++m)
#pragma unroll
      for (int n = 0; n < L::kColTiles; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = at.row + 16 * m + (e >> 1) * 8, c = c0 + at.col + 8 * n + (e & 1);
          if (r < p.d && c < p.d) last[r * p.d + c] = S[m][n][e];
        }
  }
}

// dg over one chunk of one (b, h).  With S the state that enters the chunk and D the gradient of the one that
// leaves it, dg_t = e^{g_t} <S_{t-1}, dS_t> is the sum of what has the gate between its two tokens:
//   pairs of the chunk    M_ij = scale e^{b_i - b_j} (q_i . k_j)(do_i . v_j)    j < t <= i
//   queries and S         r_i  = scale e^{b_i} q_i . S do_i                     t <= i     (dots of the scan of dq)
//   keys and D            c_j  = e^{B - b_j} k_j . D v_j                        j < t      (dots of the scan of dk)
//   both states           e^B <S, D>
// Nothing cancels: every term carries the decay of gate t, so dg is as exact as its own terms however strongly
// gates forget, a closed gate has 0, and what is not finite stays on its side.  (A running sum of q . dq - k . dk,
// which needs no pairs, has the error of all it has summed, however small dg itself.)
//
// A warp takes a group of rows i, a quarter of the chunk, and walks the tiles of 16 columns j in front of it: both dots
// on mma.sync, then sums over M's rows (for the gates of the rows' group) and over its columns (for the gates of the
// columns' group); a gate in between takes whole groups, and the pairs of one group are summed for each of its gates.
//
// q, k, v, dout and both states are read once more, so memory bounds it: bf16 gradients of [2, 16384, 70, 32] 183 us
// for 0.77 GB (4.2 TB/s), of [4, 4096, 12, 64] 45 us for 0.16 GB (3.4 TB/s): there 3.4 waves of CTAs load together, at 5 to
// 6 TB/s, and then compute together.  Not faster: chunks fetched one ahead by CTAs that stay (two stages leave an SM
// eight warps: 65 us), rows straight from memory to registers (99), eight warps of one tile (53; 229), the next wave's
// rows asked for in L2 (0.92 of the time here, 1.05 with 70 heads).
struct GateGrad {
  Operand q, k, v, dout, dg;
  const float *qdots, *kdots;    // r and c [slices][B][H][N]
  const float *enter, *leave;    // S and D of every chunk, as the scans hold them; whole: [B][H][d][d] or null for zero
  const float* sums;             // b of every chunk, high parts and low parts
  int64_t N, H, BH;
  uint32_t chunks;               // of 64 TILES tokens
  int32_t d, slices;
  float scale;
  bool whole;                    // one chunk: the call's own states
};

// A warp has TILES blocks of 16 rows, one for chunks of 64 tokens and two for those of 128.  Four warps; float32, with
// six products a term, takes four for q . k and four for do . v, which hand theirs over through shared memory.
template <typename T, int DK, int TILES>
struct GateTile {
  static constexpr int kIn = Terms<T>::kIn, kTokens = kChunk * TILES, kRows = 16 * TILES, kGroups = 4;
  static constexpr int kRoles = kIn > 1 ? 2 : 1, kThreads = 128 * kRoles;
  static constexpr int kPlane = kChunk * DK * 2;   // bytes of one term of 64 tokens
  static constexpr int kOperand = TILES * kIn * kPlane;
  static constexpr int kBytes = 4 * kOperand + (kRoles > 1 ? kGroups * (kGroups + 1) / 2 * 1024 : 0);
  // CTAs an SM holds at least: by shared memory, and by registers
  static constexpr int kFit = 227 * 1024 / (kBytes + 4608 * TILES), kMost = DK == 128 ? 2 : DK == 64 ? 4 - kRoles : kRoles > 1 ? 3 : 5;
  static constexpr int kCtas = kFit < kMost ? kFit : kMost;
};

// A warp's rows as A operands; float32's three terms stay in shared memory.
template <typename T, int DK, int TILES>
struct GroupRows {
  using L = GateTile<T, DK, TILES>;
  uint32_t x, y;
  int group, lane;
  uint32_t held[L::kIn > 1 ? 1 : TILES][L::kIn > 1 ? 1 : DK / 16][4];
  // Byte offset of 16 rows' plane and the row in it.
  static __device__ __forceinline__ uint32_t plane(int tile) { return (tile >> 2) * L::kIn * L::kPlane; }
  __device__ __forceinline__ uint32_t row_of(int tile) const { return 16 * (tile & 3) + (lane & 7) + ((lane >> 3) & 1) * 8; }
  __device__ __forceinline__ GroupRows(uint32_t x_, uint32_t y_, int group_, int lane_) : x(x_), y(y_), group(group_), lane(lane_) {
    if constexpr (L::kIn == 1)
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
          const int tile = TILES * group + i;
          ldsm(held[i][ks], x + plane(tile) + unit_at<DK>(row_of(tile), 2 * ks + (lane >> 4)));
        }
  }
  // Dots of tiles FROM .. TO - 1 of them with rows 16 s .. of y: mma accumulators of 16 by 16.
  template <int FROM, int TO>
  __device__ __forceinline__ void dots(float (&c)[TO - FROM][2][4], int s) const {
    const uint32_t from = y + plane(s);
    const int yr = 16 * (s & 3) + (lane & 7) + (lane >> 4) * 8;
    Accumulators<2, (L::kIn > 1)> acc[TO - FROM];
    if (L::kIn > 1)
#pragma unroll
      for (int i = 0; i < TO - FROM; ++i) acc[i].clear();
#pragma unroll(L::kIn > 1 ? 1 : DK / 16)
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t b[L::kIn][1][4];
#pragma unroll
      for (int t = 0; t < L::kIn; ++t) ldsm(b[t][0], from + t * L::kPlane + unit_at<DK>(yr, 2 * ks + ((lane >> 3) & 1)));
#pragma unroll
      for (int i = 0; i < TO - FROM; ++i) {
        uint32_t a[L::kIn][4];
#pragma unroll
        for (int t = 0; t < L::kIn; ++t) {
          const int tile = TILES * group + FROM + i;
          if constexpr (L::kIn > 1)
            ldsm(a[t], x + plane(tile) + t * L::kPlane + unit_at<DK>(row_of(tile), 2 * ks + (lane >> 4)));
          else
#pragma unroll
            for (int e = 0; e < 4; ++e) a[t][e] = held[FROM + i][ks][e];
        }
        mma_terms(acc[i], 0, a, b, L::kIn == 1 && ks == 0);
      }
    }
#pragma unroll
    for (int i = 0; i < TO - FROM; ++i)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[i][f][e] = acc[i].get(f, e);
  }
};

// Sums over a warp's eight lanes of its four columns, 2 (lane % 4) and the next and those eight behind; a lane gets that
// of column_of(lane).
__device__ __forceinline__ float columns_total(const float (&z)[4], int lane) {   // halves change hands until a lane pair has one
  const bool up = lane & 16, right = lane & 8;
  const float a0 = (up ? z[2] : z[0]) + __shfl_xor_sync(~0u, up ? z[0] : z[2], 16);
  const float a1 = (up ? z[3] : z[1]) + __shfl_xor_sync(~0u, up ? z[1] : z[3], 16);
  const float a = (right ? a1 : a0) + __shfl_xor_sync(~0u, right ? a0 : a1, 8);
  return a + __shfl_xor_sync(~0u, a, 4);
}
__device__ __forceinline__ int column_of(int lane) { return ((lane & 16) >> 1) + 2 * (lane & 3) + ((lane & 8) >> 3); }

__device__ __forceinline__ float dot4(const float4& f, const float4& g, float s) {
  return fmaf(f.x, g.x, fmaf(f.y, g.y, fmaf(f.z, g.z, fmaf(f.w, g.w, s))));
}

// This thread's share of <S, D>, both in the order in which a scan's threads hold them (tcgen05: two tiles a warp here).
template <int DK, int TILES, int THREADS>
__device__ __forceinline__ float states_dot(const float4* enter, const float4* leave, int d) {
  float s = 0.0f;
  if constexpr (TILES == 2) {
#pragma unroll
    for (int i = 0; i < DK * DK / 4 / THREADS; ++i) s = dot4(enter[threadIdx.x + THREADS * i], leave[threadIdx.x + THREADS * i], s);
  } else {
    const int quads = held_state<DK>(d).quads;
#pragma unroll 4
    for (int i = threadIdx.x; i < quads; i += THREADS) s = dot4(enter[i], leave[i], s);
  }
  return s;
}

template <typename T, int DK, bool ASYNC, int TILES>
__global__ void __launch_bounds__(GateTile<T, DK, TILES>::kThreads, GateTile<T, DK, TILES>::kCtas)
    gated_gate_grad(const __grid_constant__ GateGrad p) {
  using L = GateTile<T, DK, TILES>;
  constexpr int kTokens = L::kTokens, kGroups = L::kGroups, kRows = L::kRows, kThreads = L::kThreads;
  __shared__ float rows[kTokens];                       // M's rows in front of their group
  __shared__ float within[kTokens];                     // what a gate has of the pairs of its own group
  __shared__ float inner[TILES == 2 ? kTokens : 1];     // of a group's second tile with its first: columns, then rows
  __shared__ float column[kGroups][kTokens - kRows];    // M's columns in front of each group of rows
  __shared__ __align__(16) float factor[kGroups][kTokens - kRows];   // scale e^{m - b_j}, m at the group's edge
  __shared__ float r_block[kGroups], c_block[kGroups];  // r and c over a group
  __shared__ float part[kThreads / 32];                 // of <S, D>
  __shared__ __align__(16) float hi[kTokens], lo[kTokens];   // b_i
  extern __shared__ __align__(16) char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = threadIdx.x, d = p.d;
  const int group = me / kRows, unit = me % kRows;      // of the thread's token
  // Heads first: their rows of a token lie side by side in memory.  32-bit divisions.
  const uint32_t H = static_cast<uint32_t>(p.H), of_batch = blockIdx.x / H, batch = of_batch / p.chunks;
  const uint32_t chunk = of_batch - batch * p.chunks;
  const int64_t b = batch, h = blockIdx.x - of_batch * H, bh = b * p.H + h, t0 = static_cast<int64_t>(chunk) * kTokens;
  const int64_t slot = bh * p.chunks + chunk;   // of the chunk's states and sums
  const int count = static_cast<int>(min(p.N - t0, static_cast<int64_t>(kTokens)));
  auto sum_at = [&](int i) { return Sum{hi[i], lo[i]}; };
  const Sum none = {0.0f, 0.0f};

  const uint32_t first = ptx::smem_u32(smem), second = first + 2 * L::kOperand;
  if constexpr (ASYNC) {
    if (d < DK) {   // columns behind d stay zero
      for (int i = me; i < L::kBytes / 16; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
    }
    constexpr int kUnits = DK / 8, kPass = kThreads / kUnits;   // 16-byte units of a row, rows a pass
    static_assert(kPass % 8 == 0, "a pass keeps the units' places");
    const int r = me / kUnits, u = me % kUnits;
    auto fetch = [&](const Operand& o, uint32_t to) {
      const T* base = static_cast<const T*>(o.data) + (b * o.sb + h * o.sh + t0 * o.sn);
      const T* from = base + r * o.sn + 8 * u;
      to += unit_at<DK>(r, u);
      if (count == kTokens) {
#pragma unroll
        for (int i = 0; i < kTokens / kPass; ++i, from += kPass * o.sn) cp_async_16(to + i * kPass * DK * 2, from, 16);
      } else {
#pragma unroll
        for (int i = 0; i < kTokens / kPass; ++i, from += kPass * o.sn) {
          const bool in = r + i * kPass < count;
          cp_async_16(to + i * kPass * DK * 2, in ? from : base, in ? 16 : 0);
        }
      }
    };
    if (8 * u < d) {
      fetch(p.q, first);
      fetch(p.k, first + L::kOperand);
      fetch(p.dout, second);
      fetch(p.v, second + L::kOperand);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  auto load = [&](const Operand& x, const Operand& y, char* to) {   // rows that lie otherwise
    const RowLoader<T, DK, kThreads, false> of_x(x, b, h, 0, d), of_y(y, b, h, 0, d);
    load_plain(static_cast<int64_t>(chunk), p.N, PlainPart<T, DK, kThreads>{of_x, to},
               PlainPart<T, DK, kThreads>{of_y, to + L::kOperand});
  };
  // Everything else is asked for before any of it is waited for: the scans' dots and the gates' sums, a token a thread
  constexpr int kSlices = 4;   // at most
  float q_dot[kSlices] = {}, k_dot[kSlices] = {}, b_hi = 0.0f, b_lo = 0.0f;
  if (me < kTokens) {
    b_hi = p.sums[2 * kTokens * slot + me];
    b_lo = p.sums[2 * kTokens * slot + kTokens + me];
  }
  if (me < count) {
    const int64_t at = bh * p.N + t0 + me, step = p.BH * p.N;
#pragma unroll
    for (int k = 0; k < kSlices; ++k)
      if (k < p.slices) {
        q_dot[k] = p.qdots[at + k * step];
        k_dot[k] = p.kdots[at + k * step];
      }
  }
  {   // <S, D>
    float s = 0.0f;
    if (p.whole) {
      const float *x = p.enter + bh * d * d, *y = p.leave + bh * d * d;
      if (p.enter && p.leave)
        for (int i = me; i < d * d; i += kThreads) s = fmaf(x[i], y[i], s);
    } else {
      const int64_t at = slot * (TILES == 2 ? DK * DK / 4 : held_state<DK>(d).quads);
      s = states_dot<DK, TILES, kThreads>(reinterpret_cast<const float4*>(p.enter) + at, reinterpret_cast<const float4*>(p.leave) + at, d);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(~0u, s, k);
    if (lane == 0) part[warp] = s;
  }

  if constexpr (!ASYNC) {
    static_assert(TILES == 1, "a part of 64 tokens");
    load(p.q, p.k, smem);
    load(p.dout, p.v, smem + 2 * L::kOperand);
  }
  if (me < kTokens) {
    hi[me] = b_hi;
    lo[me] = b_lo;
  }
  const float r_own = (q_dot[0] + q_dot[1]) + (q_dot[2] + q_dot[3]), c_own = (k_dot[0] + k_dot[1]) + (k_dot[2] + k_dot[3]);
  if (me < kTokens) {
    float u = (lane & 1 ? c_own : r_own) + __shfl_xor_sync(~0u, lane & 1 ? r_own : c_own, 1);   // r in even lanes, c in odd ones
#pragma unroll
    for (int k = 2; k < kRows; k <<= 1) u += __shfl_xor_sync(~0u, u, k);
    if (unit < 2) (unit ? c_block : r_block)[group] = u;
  }
  if constexpr (ASYNC) asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // neighbouring CTAs give the rows that see more to different warps
  const int own = (warp + static_cast<int>(blockIdx.x)) & (kGroups - 1), row0 = kRows * own, role = warp / kGroups;
  // Pairs of two groups: e^{b_i - m} e^{m - b_j}, m at the edge of the rows' group, each factor out of one of the sums
  const Sum m = own ? sum_at(row0 - 1) : none;
  Sum at_row[TILES][2];   // of rows lane / 4 and eight behind it
  float f[TILES][2];
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      at_row[i][e] = sum_at(row0 + 16 * i + 8 * e + (lane >> 2));
      f[i][e] = exp2_of(at_row[i][e], m);
    }
  for (int j = lane; role == 0 && j < row0; j += 32) factor[own][j] = p.scale * exp2_of(m, sum_at(j));
  __syncwarp();
  Two of_row[TILES][2];   // sums over what lies in front of the group
#pragma unroll
  for (int i = 0; i < TILES; ++i) of_row[i][0] = of_row[i][1] = two(0.0f, 0.0f);
  auto pairs = [&](const float (&x)[TILES][2][4], const float (&y)[TILES][2][4], int s) {
    float z[4];
    const float* col = factor[own] + 16 * s;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const float2 w = *reinterpret_cast<const float2*>(col + 8 * g + 2 * (lane & 3));
      Two sum = two(0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const Two u = mul(two(x[i][g][2 * e], x[i][g][2 * e + 1]), two(y[i][g][2 * e], y[i][g][2 * e + 1]));
          of_row[i][e] = fma(u, two(w.x, w.y), of_row[i][e]);
          sum = i + e ? fma(u, two(f[i][e], f[i][e]), sum) : mul(u, two(f[i][e], f[i][e]));
        }
      apart(sum, z[2 * g], z[2 * g + 1]);
    }
    const float a = columns_total(z, lane);
    const int j = 16 * s + column_of(lane);
    if (!(lane & 4)) column[own][j] = factor[own][j] * a;
  };
  // Weights within a group, from the sums themselves: tile i's rows, columns 8 g + 2 (lane % 4) and the next of tile s.
  auto weigh = [&](float (&x)[2][4], const float (&y)[2][4], int i, int s, bool cut) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int j = 8 * g + 2 * (lane & 3);
      const float2 hj = *reinterpret_cast<const float2*>(hi + row0 + 16 * s + j), lj = *reinterpret_cast<const float2*>(lo + row0 + 16 * s + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = p.scale * exp2_of(at_row[i][e >> 1], e & 1 ? Sum{hj.y, lj.y} : Sum{hj.x, lj.x});
        x[g][e] = !cut || j + (e & 1) < (lane >> 2) + (e >> 1) * 8 ? x[g][e] * y[g][e] * w : 0.0f;
      }
    }
  };
  // Pairs of one tile: gate t has the sum over rows i >= t of what row i holds in front of column t.
  auto triangle = [&](const float (&x)[2][4], int i) {
    float z[4] = {};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float before[2], total = 0.0f;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float u = x[g][2 * half] + x[g][2 * half + 1];
#pragma unroll
        for (int k = 1; k < 4; k <<= 1) {
          const float o = __shfl_up_sync(~0u, u, k, 4);
          if ((lane & 3) >= k) u += o;
        }
        const float o = __shfl_up_sync(~0u, u, 1, 4);
        before[g] = (lane & 3) ? o : 0.0f;
        if (g == 0) total = __shfl_sync(~0u, u, 3, 4);
      }
      before[1] += total;
      const int r = (lane >> 2) + 8 * half, t = 2 * (lane & 3);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (r >= 8 * g + t) z[2 * g] += before[g];
        if (r >= 8 * g + t + 1) z[2 * g + 1] += before[g] + x[g][2 * half];
      }
    }
    const float a = columns_total(z, lane);
    if (!(lane & 4)) within[row0 + 16 * i + column_of(lane)] = a;
  };
  // And of a group's second tile with its first: sums over columns and over rows.
  auto square = [&](const float (&x)[2][4]) {
    const float z[4] = {x[0][0] + x[0][2], x[0][1] + x[0][3], x[1][0] + x[1][2], x[1][1] + x[1][3]};
    const float a = columns_total(z, lane);
    if (!(lane & 4)) inner[row0 + column_of(lane)] = a;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float u = (x[0][2 * e] + x[0][2 * e + 1]) + (x[1][2 * e] + x[1][2 * e + 1]);
      u += __shfl_xor_sync(~0u, u, 1);
      u += __shfl_xor_sync(~0u, u, 2);
      if ((lane & 3) == 0) inner[row0 + 16 + 8 * e + (lane >> 2)] = u;
    }
  };

  using Rows = GroupRows<T, DK, TILES>;
  float x[TILES][2][4], y[TILES][2][4];
  if constexpr (L::kRoles > 1) {
    float kept[kGroups - 1][1][2][4];   // q . k
    float4* const handed = reinterpret_cast<float4*>(smem + 4 * L::kOperand) + 32 * own * (own + 1) + lane;   // do . v
    if (role == 0) {
      const Rows q(first, first + L::kOperand, own, lane);
#pragma unroll
      for (int s = 0; s < kGroups - 1; ++s)
        if (s < own) q.template dots<0, 1>(kept[s], s);
      q.template dots<0, 1>(x, own);
    } else {
      const Rows z(second, second + L::kOperand, own, lane);
#pragma unroll 1
      for (int s = 0; s <= own; ++s) {
        z.template dots<0, 1>(y, s);
#pragma unroll
        for (int g = 0; g < 2; ++g) handed[64 * s + 32 * g] = make_float4(y[0][g][0], y[0][g][1], y[0][g][2], y[0][g][3]);
      }
    }
    __syncthreads();
    auto take = [&](int s) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float4 u = handed[64 * s + 32 * g];
        y[0][g][0] = u.x; y[0][g][1] = u.y; y[0][g][2] = u.z; y[0][g][3] = u.w;
      }
    };
    if (role == 0) {
#pragma unroll
      for (int s = 0; s < kGroups - 1; ++s)
        if (s < own) {
          take(s);
          pairs(kept[s], y, s);
        }
      take(own);
      weigh(x[0], y[0], 0, 0, true);
      triangle(x[0], 0);
    }
  } else {
    const Rows q(first, first + L::kOperand, own, lane), z(second, second + L::kOperand, own, lane);
#pragma unroll 1
    for (int s = 0; s < TILES * own; ++s) {
      q.template dots<0, TILES>(x, s);
      z.template dots<0, TILES>(y, s);
      pairs(x, y, s);
    }
    q.template dots<0, TILES>(x, TILES * own);
    z.template dots<0, TILES>(y, TILES * own);
    weigh(x[0], y[0], 0, 0, true);
    triangle(x[0], 0);
    if constexpr (TILES == 2) {
      weigh(x[1], y[1], 1, 0, false);
      square(x[1]);
      float u[1][2][4], w[1][2][4];
      q.template dots<1, 2>(u, 2 * own + 1);
      z.template dots<1, 2>(w, 2 * own + 1);
      weigh(u[0], w[0], 1, 1, true);
      triangle(u[0], 1);
    }
  }
  if (role == 0)
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float u, w;
      apart(of_row[i][e], u, w);
      u += w;
      u += __shfl_xor_sync(~0u, u, 1);
      u += __shfl_xor_sync(~0u, u, 2);
      if ((lane & 3) == 0) rows[row0 + 16 * i + 8 * e + (lane >> 2)] = f[i][e] * u;
    }
  __syncthreads();
  if (me >= kTokens) return;
  // what every gate of the group has (both states, whole groups on both sides), a share a lane: a gate meets the shares
  // from its lane on in r's sum, those in front in c's
  float share = 0.0f;
  if (unit < kGroups) {
    share = exp2_of(sum_at(kTokens - 1), none) * (L::kRoles > 1 ? part[unit] + part[kGroups + unit] : part[unit]);
    if (unit > group) share += r_block[unit];
    if (unit < group) share += c_block[unit];
  }
#pragma unroll
  for (int i = 2; i < kGroups; ++i)
#pragma unroll
    for (int j = 0; j < i - 1; ++j)
      if (i > group && group > j) share += column[i][kRows * j + unit];
  // rows from the gate's on and columns in front of it within the group
  float r = r_own + rows[me] + share, c = c_own + share;
#pragma unroll
  for (int i = 1; i < kGroups; ++i)
    if (i > group) c += column[i][me];
#pragma unroll
  for (int k = 1; k < kRows; k <<= 1) {
    const float u = __shfl_down_sync(~0u, r, k, kRows), w = __shfl_up_sync(~0u, c, k, kRows);
    if (unit + k < kRows) r += u;
    if (unit >= k) c += w;
  }
  const float in_front = __shfl_up_sync(~0u, c, 1, kRows);
  float dg = within[me] + r + (unit ? in_front : 0.0f);
  if constexpr (TILES == 2) {   // the first tile's gates: columns in front; the second's: rows from the gate's on
    const bool back = unit >= 16;
    float u = inner[me];
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) {
      const float o = __shfl_sync(~0u, u, back ? lane + k : lane - k);
      if (back ? lane + k < 32 : lane >= k) u += o;
    }
    const float o = __shfl_up_sync(~0u, u, 1);
    dg += back ? u : lane ? o : 0.0f;
  }
  if (me < count) from_f(static_cast<T*>(p.dg.data) + b * p.dg.sb + h * p.dg.sh + (t0 + me) * p.dg.sn, dg);
}

// ------------------------------------------------------------------ launches

int padded(int32_t d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }

// CTAs of gated_scan an SM holds.  (float32 [2, 3000, 10, 32] gradients: two 111 us, three 92, four 95.)
int ctas_an_sm(const GatedProblem& p) {
  if (p.d > 64) return 1;
  return p.dtype == MHLA_BF16 || p.d <= 32 ? 3 : 2;
}

// As many spans as one wave of CTAs takes: a few beyond it cost a second wave (float32 [3, 5181, 4, 64],
// 324 CTAs on 304 places 127 us, 300 CTAs 96).
Cut cut_for(const GatedProblem& p, int scans) {
  Cut c;
  c.chunks = (p.N + kChunk - 1) / kChunk;
  const int64_t have = p.B * p.H * (p.d > 64 ? 2 : 1) * scans;
  const int64_t room = int64_t{kSms} * ctas_an_sm(p);
  int64_t spans = std::max<int64_t>(1, room / have);
  c.span_chunks = (c.chunks + spans - 1) / spans;
  c.spans = (c.chunks + c.span_chunks - 1) / c.span_chunks;
  return c;
}

// 16-byte rows: cp.async takes them as they lie.
bool rows_of_16(const GatedProblem& p, std::initializer_list<const Operand*> os) {
  if (p.dtype != MHLA_BF16 || p.d % 8 != 0) return false;
  for (const Operand* o : os)
    if (reinterpret_cast<uintptr_t>(o->data) % 16 != 0 || o->sb % 8 != 0 || o->sn % 8 != 0 || o->sh % 8 != 0)
      return false;
  return true;
}

template <typename T, int DK, bool ASYNC>
int launch_span_state(const ScanSet& set, int scans, cudaStream_t s) {
  using L = Tile<T, DK, ASYNC>;
  constexpr int kBytes = L::kStages * L::kIn * (L::kK + L::kV);
  // a per-device setting: made on every call, for whichever device is current
  if (cudaFuncSetAttribute(gated_span_state<T, DK, ASYNC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) !=
      cudaSuccess)
    return MHLA_ERR_CUDA;
  const int64_t slices = (set.d + L::DV - 1) / L::DV;
  KernelTimer timer("gated_span_state", s);
  gated_span_state<T, DK, ASYNC>
      <<<dim3(static_cast<unsigned>(set.BH * slices * (set.spans - 1)), scans), L::kThreads, kBytes, s>>>(set);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, bool ASYNC, bool GRAD>
int launch_scan(const ScanSet& set, int scans, cudaStream_t s) {
  using L = Tile<T, DK, ASYNC>;
  constexpr int kBytes = ScanShared<T, DK, ASYNC>::kBytes;
  if (cudaFuncSetAttribute(gated_scan<T, DK, ASYNC, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) !=
      cudaSuccess)
    return MHLA_ERR_CUDA;
  const int64_t slices = (set.d + L::DV - 1) / L::DV;
  KernelTimer timer("gated_scan", s);
  gated_scan<T, DK, ASYNC, GRAD><<<dim3(static_cast<unsigned>(set.BH * slices * set.spans), scans), L::kThreads, kBytes, s>>>(set);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, bool ASYNC>
int run_scan_kernel(const ScanSet& set, int scans, bool span_state, cudaStream_t s) {
  if (span_state) return launch_span_state<T, DK, ASYNC>(set, scans, s);
  return scans > 1 ? launch_scan<T, DK, ASYNC, true>(set, scans, s) : launch_scan<T, DK, ASYNC, false>(set, scans, s);
}

template <typename T, bool ASYNC>
int run_scans_as(const ScanSet& set, int scans, bool span_state, cudaStream_t s) {
  switch (padded(set.d)) {
    case 32: return run_scan_kernel<T, 32, ASYNC>(set, scans, span_state, s);
    case 64: return run_scan_kernel<T, 64, ASYNC>(set, scans, span_state, s);
    default: return run_scan_kernel<T, 128, ASYNC>(set, scans, span_state, s);
  }
}

// One scan is the forward, three are the gradients.
int run_scans(const GatedProblem& p, const ScanSet& set, int scans, bool async, bool span_state, cudaStream_t s) {
  if (p.dtype == MHLA_F32) return run_scans_as<float, false>(set, scans, span_state, s);
  return async ? run_scans_as<__nv_bfloat16, true>(set, scans, span_state, s)
               : run_scans_as<__nv_bfloat16, false>(set, scans, span_state, s);
}

int run_join(const ScanSet& set, int scans, cudaStream_t s) {
  KernelTimer timer("gated_join", s);
  const int64_t n = set.BH * set.d * set.d;
  gated_join<<<dim3(static_cast<unsigned>((n + 255) / 256), scans), 256, 0, s>>>(set);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, bool ASYNC, int TILES>
int launch_gate_grad(const GateGrad& g, cudaStream_t s) {
  using L = GateTile<T, DK, TILES>;
  if (cudaFuncSetAttribute(gated_gate_grad<T, DK, ASYNC, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return MHLA_ERR_CUDA;
  KernelTimer timer("gated_gate_grad", s);
  gated_gate_grad<T, DK, ASYNC, TILES><<<static_cast<unsigned>(g.BH * g.chunks), L::kThreads, L::kBytes, s>>>(g);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, bool ASYNC>
int run_gate_grad_as(const GateGrad& g, cudaStream_t s) {
  switch (padded(g.d)) {
    case 32: return launch_gate_grad<T, 32, ASYNC, 1>(g, s);
    case 64: return launch_gate_grad<T, 64, ASYNC, 1>(g, s);
    default: return launch_gate_grad<T, 128, ASYNC, 1>(g, s);
  }
}

// tc: behind the tcgen05 scans, whose chunks are of 128 tokens.
int run_gate_grad(const GatedProblem& p, const GateGrad& g, bool tc, bool async, cudaStream_t s) {
  if (tc) return p.d <= 32 ? launch_gate_grad<__nv_bfloat16, 32, true, 2>(g, s) : launch_gate_grad<__nv_bfloat16, 64, true, 2>(g, s);
  if (p.dtype == MHLA_F32) return run_gate_grad_as<float, false>(g, s);
  return async ? run_gate_grad_as<__nv_bfloat16, true>(g, s) : run_gate_grad_as<__nv_bfloat16, false>(g, s);
}

ScanSet scan_set(const GatedProblem& p, const Cut& c) {
  ScanSet s = {};
  s.g = p.g;
  s.N = p.N; s.H = p.H; s.BH = p.B * p.H;
  s.span_chunks = c.span_chunks; s.chunks = c.chunks;
  s.spans = static_cast<int32_t>(c.spans);
  s.d = p.d;
  return s;
}

Scan plain_scan(const Operand& q, const Operand& k, const Operand& v, const Operand& out) {
  Scan a = {};
  a.q = q; a.k = k; a.v = v; a.out = out;
  a.out_scale = a.state_scale = a.k_scale = 1.0f;
  a.init_spans = 1;
  return a;
}

struct SpanBuffers {
  float *local, *decay;
};

size_t span_bytes(const GatedProblem& p, const Cut& c) {
  if (c.spans < 2) return 0;
  const int64_t n = p.B * p.H * c.spans;
  return align_up(static_cast<size_t>(n * p.d * p.d) * 4) + align_up(static_cast<size_t>(n) * 4);
}

// Enough for either kernel, whichever takes the call's operands.
size_t most_span_bytes(const GatedProblem& p, int scans) {
  const size_t n = span_bytes(p, cut_for(p, scans));
  return tc_supported(p) ? std::max(n, span_bytes(p, tc_cut(p, scans))) : n;
}

// Parts of the columns whose dots are summed apart: by gated_scan, the most of either kernel.
int scan_dot_slices(const GatedProblem& p) { return p.d > 64 ? 4 : 1; }
int64_t dot_slices(const GatedProblem& p) { return std::max(scan_dot_slices(p), p.d > 32 ? 2 : 1); }

size_t dot_bytes(const GatedProblem& p) { return align_up(static_cast<size_t>(dot_slices(p) * p.B * p.H * p.N) * 4); }

// The state that enters each chunk (of 64 tokens, or 128 of the tcgen05 scan), and the gates' sums in each.
// A sequence of one chunk has the call's own states at both ends.
size_t entry_bytes(const GatedProblem& p, bool tc) {
  const int chunk = tc ? kTcChunk : kChunk, side = padded(p.d);
  if (p.N <= chunk) return 0;
  const int quads = tc ? side * side / 4 : side == 32 ? held_state<32>(p.d).quads : held_state<64>(p.d).quads;
  return align_up(static_cast<size_t>(p.B * p.H * ((p.N + chunk - 1) / chunk)) * quads * 16);
}
size_t sum_bytes(const GatedProblem& p, int chunk) {
  return align_up(static_cast<size_t>(p.B * p.H * ((p.N + chunk - 1) / chunk) * chunk) * 8);
}

SpanBuffers carve_spans(const GatedProblem& p, const Cut& c, char** base) {
  if (c.spans < 2) return SpanBuffers{nullptr, nullptr};
  const int64_t n = p.B * p.H * c.spans;
  SpanBuffers s;
  s.local = reinterpret_cast<float*>(*base);
  *base += align_up(static_cast<size_t>(n * p.d * p.d) * 4);
  s.decay = reinterpret_cast<float*>(*base);
  *base += align_up(static_cast<size_t>(n) * 4);
  return s;
}

// The kernels of one call: tcgen05 where the operands suit it, else mma.sync.
struct Runner {
  const GatedProblem& p;
  bool tc, async;
  TcMaps maps;
  cudaStream_t s;
  int run(const ScanSet& set, int scans, bool span_state) const {
    return tc ? launch_tc_scan(set, maps, scans, span_state, s) : run_scans(p, set, scans, async, span_state, s);
  }
};

// Which kernel takes operands that suit both.  tcgen05 runs one CTA an SM at half to a third of
// mma.sync's time a token, but starts slowly (6 us a wave of CTAs) and cuts long sequences of
// few heads into fewer, longer spans.  Measured, mma.sync against tcgen05 in us:
//   up to 384 tokens, one wave         d 64, 48 heads x 256 forwards: 18.4, 10.1;   d 32: 11.5, 8.7
//   longer, d > 32: enough tokens      16 heads x 2048: 25.6, 21.9;   1 x 16384: 35.5, 23.5;   4 x 1024: 15.5, 18.5
//   longer, d <= 32: whole sequences   128 heads x 1024: 35.0, 20.7;   48 x 1024 (two launches): 17.8, 20.5
//   several waves: enough chunks each  d 64, 512 x 256: 47.8, 37.9;  512 x 128: 28.2, 29.5;
//                                      d 32, 512 x 1024: 92.0, 76.2;  512 x 512: 43.8, 47.4
bool wants_tc(const GatedProblem& p, int scans) {
  if (!tc_supported(p) || p.N < 128) return false;
  const int64_t ctas = p.B * p.H * scans;
  if (ctas > kSms) return p.N >= (p.d <= 32 ? 1024 : 256);
  if (p.N <= 384) return true;
  return p.d <= 32 ? 2 * ctas > kSms : ctas * p.N >= 16384;
}

}  // namespace

size_t gated_workspace_bytes(const GatedProblem& p) { return most_span_bytes(p, 1); }

size_t gated_bwd_workspace_bytes(const GatedProblem& p) {
  return 2 * most_span_bytes(p, 3) + 2 * dot_bytes(p) +
         2 * std::max(entry_bytes(p, false), tc_supported(p) ? entry_bytes(p, true) : 0) +
         std::max(sum_bytes(p, kChunk), sum_bytes(p, kTcChunk));
}

int launch_gated_forward(const GatedProblem& p, const float* state_in, const Operand& out, float* state_out,
                         void* workspace, void* stream) {
  Scan a = plain_scan(p.q, p.k, p.v, out);
  a.out_scale = a.state_scale = p.scale;
  a.init = state_in;
  a.last = state_out;
  Runner r{p, false, rows_of_16(p, {&p.q, &p.k, &p.v, &out}), {}, static_cast<cudaStream_t>(stream)};
  ScanSet set = {};
  set.scan[0] = a;
  r.tc = r.async && wants_tc(p, 1) && tc_maps(p, set, 1, &r.maps);
  const Cut c = r.tc ? tc_cut(p, 1) : cut_for(p, 1);
  set = scan_set(p, c);
  char* base = static_cast<char*>(workspace);
  const SpanBuffers sb = carve_spans(p, c, &base);
  a.local = sb.local;
  a.decay = sb.decay;
  set.scan[0] = a;
  if (c.spans > 1) {
    int rc = r.run(set, 1, true);
    // A few spans are joined by the scan as it starts: a launch for it costs 4 us, a span's
    // loads from L2 0.7.  Not when the last span's CTA writes the state that the others would read.
    const bool join = r.tc && c.spans <= 6 && (!state_in || state_out != state_in);
    if (rc == MHLA_OK && !join) rc = run_join(set, 1, r.s);
    if (rc != MHLA_OK) return rc;
    set.scan[0].join = join;
    if (!join) {
      set.scan[0].init = sb.local;
      set.scan[0].init_spans = set.spans;
    }
  }
  return r.run(set, 1, false);
}

int launch_gated_backward(const GatedProblem& p, const GatedBackward& b, void* workspace, void* stream) {
  Scan dq = plain_scan(b.dout, p.v, p.k, b.dq);   // its state: S^T
  dq.out_scale = dq.state_scale = p.scale;
  dq.init = b.state_in;
  dq.init_transposed = 1;
  dq.dot = p.q;
  Scan dk = plain_scan(p.v, b.dout, p.q, b.dk);   // its state: dS^T
  dk.reverse = 1;
  dk.out_scale = dk.k_scale = p.scale;
  dk.init = b.dstate_out;
  dk.init_transposed = 1;
  dk.dot = p.k;
  Scan dv = plain_scan(p.k, p.q, b.dout, b.dv);   // its state: dS
  dv.reverse = 1;
  dv.out_scale = dv.k_scale = p.scale;
  dv.init = b.dstate_out;
  dv.last = b.dstate_in;

  Runner r{p, false, rows_of_16(p, {&p.q, &p.k, &p.v, &b.dout, &b.dq, &b.dk, &b.dv}), {},
           static_cast<cudaStream_t>(stream)};
  ScanSet set = {};
  set.scan[0] = dq; set.scan[1] = dk; set.scan[2] = dv;
  r.tc = r.async && wants_tc(p, 3) && tc_maps(p, set, 3, &r.maps);
  const Cut c = r.tc ? tc_cut(p, 3) : cut_for(p, 3);
  char* base = static_cast<char*>(workspace);
  const SpanBuffers fwd = carve_spans(p, c, &base), back = carve_spans(p, c, &base);
  auto take = [&](size_t bytes) {
    float* at = reinterpret_cast<float*>(base);
    base += bytes;
    return at;
  };
  dq.dots = take(dot_bytes(p));
  dk.dots = take(dot_bytes(p));
  const int chunk = r.tc ? kTcChunk : kChunk;
  const bool whole = c.chunks == 1;
  if (!whole) dq.entries = take(entry_bytes(p, r.tc));
  if (!whole) dk.entries = take(entry_bytes(p, r.tc));
  dq.sums = take(sum_bytes(p, chunk));

  set = scan_set(p, c);
  dq.local = fwd.local;
  dq.decay = fwd.decay;
  dk.local = back.local;
  dk.decay = back.decay;
  set.scan[0] = dq; set.scan[1] = dk; set.scan[2] = dv;
  int rc = MHLA_OK;
  if (c.spans > 1) {
    rc = r.run(set, 2, true);
    if (rc == MHLA_OK) rc = run_join(set, 2, r.s);
    set.scan[0].init = fwd.local;
    set.scan[1].init = set.scan[2].init = back.local;
    set.scan[0].init_transposed = set.scan[1].init_transposed = 0;
    set.scan[2].init_transposed = 1;
    for (Scan& a : set.scan) a.init_spans = set.spans;
  }
  if (rc == MHLA_OK) rc = r.run(set, 3, false);
  if (rc != MHLA_OK) return rc;
  GateGrad gg = {};
  gg.q = p.q; gg.k = p.k; gg.v = p.v; gg.dout = b.dout;
  gg.dg = b.dg;
  gg.sums = dq.sums;
  gg.qdots = dq.dots; gg.kdots = dk.dots;
  gg.whole = whole;
  gg.enter = whole ? b.state_in : dq.entries;
  gg.leave = whole ? b.dstate_out : dk.entries;
  gg.N = p.N; gg.H = p.H; gg.BH = p.B * p.H; gg.chunks = static_cast<uint32_t>(c.chunks);
  gg.d = p.d;
  gg.slices = r.tc ? static_cast<int32_t>(dot_slices(p)) : scan_dot_slices(p);
  gg.scale = p.scale;
  return run_gate_grad(p, gg, r.tc, r.async, r.s);
}

// ------------------------------------------------------------------ one token

// A CTA takes one (b, h).  The state is read and written once and nothing else is of
// size, so HBM bounds it and the loads count: VEC 4 keeps four 16-byte loads of a thread in flight (d = 64),
// row groups meeting in shared memory for o.  VEC 1 takes any d and alignment.  64 sequences of 12
// heads, d = 64 (25 MB): 5.7 us, 4.5 TB/s; one sequence 3 us, a launch.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) gated_step(const GatedProblem p, float* state, const Operand out) {
  constexpr int kBatch = 4;
  __shared__ float sq[128], sk[128];
  __shared__ float part[256 * VEC];
  const int64_t bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
  auto at = [&](const Operand& o) { return static_cast<T*>(o.data) + b * o.sb + h * o.sh; };
  const int d = p.d, units = d / VEC, groups = 256 / units;   // threads a row, rows at once
  const int x = threadIdx.x % units, y = threadIdx.x / units;
  float* S = state + bh * d * d + x * VEC;
  float s[kBatch][VEC];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * groups;
      if (r >= d) continue;
      if constexpr (VEC == 4) {
        const float4 f = *reinterpret_cast<const float4*>(S + r * d);
        s[i][0] = f.x; s[i][1] = f.y; s[i][2] = f.z; s[i][3] = f.w;
      } else {
        s[i][0] = S[r * d];
      }
    }
  };
  if (y < groups) load(y);
  if (threadIdx.x < d) {
    sq[threadIdx.x] = to_f(at(p.q)[threadIdx.x]);
    sk[threadIdx.x] = to_f(at(p.k)[threadIdx.x]);
  }
  const float g = to_f(*at(p.g));
  const float decay = expf(g < kLowestGate ? kLowestGate : g);
  float v[VEC], o[VEC] = {};
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = to_f(at(p.v)[x * VEC + e]);
  __syncthreads();
  if (y < groups)
    for (int r0 = y; r0 < d; r0 += kBatch * groups) {
      if (r0 != y) load(r0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * groups;
        if (r >= d) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[i][e] = fmaf(sk[r], v[e], decay * s[i][e]);
          o[e] = fmaf(sq[r], s[i][e], o[e]);
        }
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(S + r * d) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        else
          S[r * d] = s[i][0];
      }
    }
  if (y < groups)
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[y * d + x * VEC + e] = o[e];
  __syncthreads();
  if (threadIdx.x < d) {
    float sum = 0.0f;
    for (int i = 0; i < groups; ++i) sum += part[i * d + threadIdx.x];
    from_f(at(out) + threadIdx.x, p.scale * sum);
  }
}

int launch_gated_step(const GatedProblem& p, float* state, const Operand& out, void* stream) {
  KernelTimer timer("gated_step", stream);
  const unsigned grid = static_cast<unsigned>(p.B * p.H);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool vec = p.d % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
  if (p.dtype == MHLA_BF16) {
    if (vec)
      gated_step<__nv_bfloat16, 4><<<grid, 256, 0, s>>>(p, state, out);
    else
      gated_step<__nv_bfloat16, 1><<<grid, 256, 0, s>>>(p, state, out);
  } else {
    if (vec)
      gated_step<float, 4><<<grid, 256, 0, s>>>(p, state, out);
    else
      gated_step<float, 1><<<grid, 256, 0, s>>>(p, state, out);
  }
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

}  // namespace mhla
