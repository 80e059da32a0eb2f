// The scans of gated causal linear attention (gated_kernels.cu states the recurrence)
// on the fifth-generation tensor cores: bf16, d <= 64, chunks of 128 tokens.
//
// A persistent CTA per SM walks a span of chunks.  Per chunk, b_i the sum of the log
// decays up to token i (backwards: of those behind it) and B of all of them:
//   scores  S1 = Q K^T                                128 x 128, in tensor memory
//   P_ij    = scale e^{b_i - b_j} S1_ij for j <= i    two bf16 terms, over S1 in tensor memory
//   O1      = Q S                                     S the state, two bf16 terms in shared memory
//   O2      = P V                                     A from tensor memory
//   o_i     = scale e^{b_i} O1_i + O2_i
//   L       = (e^{B - b_j} k_j)^T V                   three bf16 terms in shared memory
//   S       <- e^B S + L                              float32 in registers, rounded to nearest
// The tensor core has four times mma.sync's rate and takes its operands without
// instructions of the warps, which leaves them the splitting into terms: that work
// bounds the kernel, so twenty-four warps share it, eight for each of three steps that
// run on different chunks at once: S1 into P (score warps); k scaled and split, and the state
// (state warps); the outputs (output warps).  Two warps issue the MMAs and
// the loads (TMA, three stages), two prepare the gates.  A thread of a score or output warp
// owns a row, so a row's factor is a register and the columns' factors are read by broadcast.
//
// Measured, all launches: bf16 [4, 4096, 12, 64] forward 54 us, gradients 153; [4, 65536, 6, 64] forward
// 330 us; [2, 16384, 70, 32] gradients 1113 us.  A chunk takes an SM 2.6 us (forward) to 3.4 (gradients) where HBM would
// need 1.5, and no rate is reached (issue slots 50 to 60%, tensor pipe 25%, HBM 30%): five hand-overs a
// chunk, each with a split into terms behind it, are a chain.  Not faster: equal shares of k's rows for two roles (1.1x), waits that sleep
// (1.0 to 1.05x), one waiting lane a warp (1.5x), terms left out (0.94x, and less exact).
//
// Every wait is bounded; one that gives up sets bit 0 of this file's error
// word and an abort flag, the CTA drains what it issued and releases tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "gated_common.cuh"
#include "mhla_internal.h"
#include "ptx.cuh"
#include "tc_common.cuh"
#include "tma_host.h"

namespace mhla {

__device__ unsigned int g_gated_error = 0;

namespace gated {
namespace {

using namespace tc;

constexpr int kScoreWarps = 8, kStateWarps = 8, kOutWarps = 8;   // in this order
constexpr int kFirstOut = kScoreWarps + kStateWarps, kIssuer = kFirstOut + kOutWarps, kAdder = kIssuer + 1, kGates = kIssuer + 2;   // two of these
constexpr int kThreads = 32 * (kGates + 2);
constexpr int kTileBytes = kTcChunk * 128;   // 128 rows of 64 channels, 128-byte swizzle
constexpr int kPlane = kTileBytes;           // one term of the scaled k
constexpr int kStatePlane = 64 * 128;        // one term of the state
constexpr uint32_t kSbo = 1024;              // between groups of eight rows

// Tensor memory columns.
constexpr uint32_t kScores = 0;   // two buffers of 128: S1, then P
constexpr uint32_t kO1 = 256, kO2 = 320, kL = 384;
constexpr uint32_t kTmemColumns = 512;

// What a chunk needs of its gates; blocks of 32 rows see other blocks' tokens through
// e^{b_i - m} e^{m - b_j}, m at the block's edge towards them, neither factor above 1.
struct ChunkGates {
  float hi[kTcChunk], lo[kTcChunk];   // b_i
  float row[kTcChunk];                // e^{b_i - m}
  float col[4][kTcChunk];             // out_scale e^{m - b_j}, per block of rows (its own tokens too)
  float addw[kTcChunk];               // k_scale e^{B - b_j}
  float enter[4];                     // state_scale e^m
  float total;                        // e^B
  uint32_t steep;                     // bit of a block: e^{m - b_j} of its own tokens may be large
  float pad[2];
};

// Of those, what a span's own state needs.
struct StateGates {
  float addw[kTcChunk];
  float total;
  float pad[3];
};

struct Bars {
  uint64_t full[5], freed[5], gates[8], gates_freed[8];
  uint64_t scores[2], p_ready[2];
  uint64_t state_read, out_done, out_read, k_ready[2], half_done[2], l_done[2], s_ready, fin[2];
};

struct Control {
  Bars bars;
  uint32_t tmem, abort;
  uint32_t bad;   // v held an infinity or NaN
  Sum decay[2];   // of the span, in two parts
};

template <bool ONLY_STATE>
struct Layout {
  static constexpr int kTiles = ONLY_STATE ? 2 : 3;   // q, k, v  |  k, v
  static constexpr int kStages = ONLY_STATE ? 5 : 3, kGateRing = ONLY_STATE ? 8 : 4;
  using Gates = typename std::conditional<ONLY_STATE, StateGates, ChunkGates>::type;
  static constexpr int kStage = kTiles * kTileBytes;
  static constexpr int kKp = kStages * kStage;
  static constexpr int kS = kKp + 3 * kPlane;
  static constexpr int kGates = kS + (ONLY_STATE ? 0 : 2 * kStatePlane);
  static constexpr int kControl = kGates + kGateRing * static_cast<int>(sizeof(Gates));
  static constexpr size_t kBytes = kControl + sizeof(Control) + 1024;
};
static_assert(Layout<false>::kBytes <= 227 * 1024 && Layout<true>::kBytes <= 227 * 1024, "shared memory of one CTA");

// A wait whose first look failed: bounded like tc::wait_bounded_on, the diagnostic hook
// (stall_hook.cuh) looked at before the next poll.
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, volatile uint32_t* abortf) {
  if (stall_this_warp()) {
    stalled_wait(abortf);
    *abortf = 1u;
    atomicOr(&g_gated_error, 1u);
    return false;
  }
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1; it < kWaitLimitPolls; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abortf) return false;
      if (globaltimer() - t0 > kWaitLimitNs) break;
    }
  }
  *abortf = 1u;
  atomicOr(&g_gated_error, 1u);
  return false;
}

// Every lane waits, then the warp agrees; the first look is in place.
__device__ __forceinline__ bool gwarp_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abortf) {
  bool ok = mbar_try_wait(bar, parity & 1u);
  if (!ok) ok = wait_longer(bar, parity & 1u, abortf);
  return __all_sync(0xffffffffu, ok);
}

// One lane of the warp, the same one for as long as all take part.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Lets the next grid on the stream, if it was launched with programmatic serialization, start as
// soon as every CTA of this one has come here; it still waits (ptx::grid_dep_wait) for what this one writes.
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// D (+)= A[tensor memory] B[shared memory].
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 lanes by 32 columns, spread over the warp like an mma accumulator: value 4 n + e is
// row lane / 4 + 8 (e / 2), column 8 n + 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Byte offset of a 16-byte unit of a 128-byte row in the 128-byte swizzle.
__device__ __forceinline__ int unit_at(int row, int unit) { return row * 128 + ((unit ^ (row & 7)) << 4); }

// A lane's four gates of a chunk (tokens 4 lane ..); 0 behind the end.
__device__ __forceinline__ float4 load_gates(const ScanSet& p, int64_t b, int64_t h, int64_t chunk, int lane) {
  const int64_t t = chunk * kTcChunk + 4 * lane;
  const __nv_bfloat16* g = static_cast<const __nv_bfloat16*>(p.g.data) + b * p.g.sb + h * p.g.sh + t * p.g.sn;
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = t + e < p.N ? to_f(g[e * p.g.sn]) : 0.0f;
  return make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ Sum shfl_sum(Sum s, int lane) {
  Sum r;
  r.hi = __shfl_sync(~0u, s.hi, lane);
  r.lo = __shfl_sync(~0u, s.lo, lane);
  return r;
}

// One warp: the running sums and the weights of a chunk (ONLY_STATE: those of the state alone).  Returns B.
template <bool ONLY_STATE>
__device__ __forceinline__ Sum chunk_gates(float4 g, typename Layout<ONLY_STATE>::Gates& out, const Scan& a, int lane,
                                           float* sums) {
  const Sum none = {0.0f, 0.0f}, gs[4] = {gate_sum(g.x), gate_sum(g.y), gate_sum(g.z), gate_sum(g.w)};
  const bool reverse = a.reverse;
  Sum at[4], run;
  if (reverse) {
    at[3] = none;
    at[2] = gs[3];
    at[1] = add(gs[2], at[2]);
    at[0] = add(gs[1], at[1]);
    run = add(gs[0], at[0]);
  } else {
    at[0] = gs[0];
    at[1] = add(at[0], gs[1]);
    at[2] = add(at[1], gs[2]);
    run = at[3] = add(at[2], gs[3]);
  }
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    Sum o;
    o.hi = reverse ? __shfl_down_sync(~0u, run.hi, s) : __shfl_up_sync(~0u, run.hi, s);
    o.lo = reverse ? __shfl_down_sync(~0u, run.lo, s) : __shfl_up_sync(~0u, run.lo, s);
    if (reverse ? lane + s < 32 : lane >= s) run = add(o, run);
  }
  const Sum all = shfl_sum(run, reverse ? 0 : 31);
  Sum next;   // of the lanes in front (behind)
  next.hi = reverse ? __shfl_down_sync(~0u, run.hi, 1) : __shfl_up_sync(~0u, run.hi, 1);
  next.lo = reverse ? __shfl_down_sync(~0u, run.lo, 1) : __shfl_up_sync(~0u, run.lo, 1);
  if (lane == (reverse ? 31 : 0)) next = none;
#pragma unroll
  for (int e = 0; e < 4; ++e) at[e] = add(next, at[e]);
  const int block = lane >> 3;
  auto put = [&](float* to, const float (&x)[4]) {
    reinterpret_cast<float4*>(to)[lane] = make_float4(x[0], x[1], x[2], x[3]);
  };
  if constexpr (ONLY_STATE) {
    float addw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) addw[e] = a.k_scale * exp2_of(all, at[e]);
    put(out.addw, addw);
    if (lane == 0) out.total = exp2_of(all, none);
  } else {
  // at the edge of each block of rows towards what it sees
  Sum edge[4] = {shfl_sum(run, reverse ? 8 : 0), shfl_sum(run, reverse ? 16 : 7), shfl_sum(run, reverse ? 24 : 15), shfl_sum(run, 23)};
  edge[reverse ? 3 : 0] = none;
  Sum m = edge[0];
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (block == i) m = edge[i];
  float hi[4], lo[4], row[4], addw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    hi[e] = at[e].hi;
    lo[e] = at[e].lo;
    row[e] = exp2_of(at[e], m);
    addw[e] = a.k_scale * exp2_of(all, at[e]);
  }
  put(out.hi, hi);
  put(out.lo, lo);
  if (sums) {
    put(sums, hi);
    put(sums + kTcChunk, lo);
  }
  put(out.row, row);
  put(out.addw, addw);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (reverse ? block < r : block > r) continue;   // tokens the rows of block r do not see
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = a.out_scale * exp2_of(edge[r], at[i]);
    put(out.col[r], c);
  }
  if ((lane & 7) == 0) out.enter[block] = a.state_scale * exp2_of(m, none);
  // beyond 2^40 within a block its own scores take each difference by itself
  bool far = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) far = far || !(fabsf((at[e].hi - m.hi) + (at[e].lo - m.lo)) <= 40.0f);
  const uint32_t lanes = __ballot_sync(~0u, far);
  if (lane == 0) {
    out.total = exp2_of(all, none);
    uint32_t steep = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) steep |= (lanes >> (8 * r) & 0xFFu) ? 1u << r : 0u;
    out.steep = steep;
  }
  }
  return all;
}

// Elements of the state that enters a span: init's, or (join) the state that enters the sequence
// carried through the spans in front, whose own contributions lie in local.  place(i, r, c)
// gives the i-th element's row and column, or false; a span's loads are in flight together.
template <int COUNT, typename Place>
__device__ __forceinline__ void entering(float (&S)[COUNT], const Scan& a, int64_t bh, int64_t span, int32_t spans, int d,
                                         Place place) {
  const int64_t dd = static_cast<int64_t>(d) * d;
  const float* in = a.init ? a.init + (bh * a.init_spans + (a.init_spans > 1 ? span : 0)) * dd : nullptr;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    int r, c;
    S[i] = place(i, r, c) && in ? in[a.init_transposed ? c * d + r : r * d + c] : 0.0f;
  }
  if (!a.join) return;
  const float* local = a.local + bh * spans * dd;
#pragma unroll 1
  for (int64_t s = 0; s < span; ++s, local += dd) {
    const float decay = a.decay[bh * spans + s];
    float l[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) {
      int r, c;
      l[i] = place(i, r, c) ? local[r * d + c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < COUNT; ++i) S[i] = fmaf(decay, S[i], l[i]);
  }
}

// A whole span again, token by token without the tensor core: for a span whose v held an
// infinity or NaN, which the masked products (0 times it) carried to earlier rows of its chunk (the states and the
// dots do not meet them).  Rare and slow; called once, behind the pipeline, so that it costs that no registers.
__device__ __noinline__ void redo_span(const ScanSet& p, const Scan& a, uint8_t* smem, int64_t bh, int64_t span,
                                       int64_t t0, int64_t t1) {
  float* q = reinterpret_cast<float*>(smem);
  float *k = q + 64, *v = k + 64, *part = v + 64;   // part: [8][64]
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6, d = p.d;
  const int64_t b = bh / p.H, h = bh % p.H;
  auto at = [&](const Operand& o, int64_t t) {
    return static_cast<__nv_bfloat16*>(o.data) + b * o.sb + t * o.sn + h * o.sh;
  };
  float S[8];   // rows 8 g .. of column c
  entering(S, a, bh, span, p.spans, d, [&](int i, int& r, int& col) {
    r = 8 * g + i;
    col = c;
    return r < d && c < d;
  });
#pragma unroll 1
  for (int64_t i = 0; i < t1 - t0; ++i) {
    const int64_t t = a.reverse ? t1 - 1 - i : t0 + i;
    __syncthreads();
    if (threadIdx.x < 64) {
      q[c] = c < d ? to_f(at(a.q, t)[c]) : 0.0f;
      k[c] = c < d ? a.k_scale * to_f(at(a.k, t)[c]) : 0.0f;
      v[c] = c < d ? to_f(at(a.v, t)[c]) : 0.0f;
    }
    const float gate = to_f(*at(p.g, t)), decay = expf(gate < kLowestGate ? kLowestGate : gate);
    __syncthreads();
    if (g < 8) {
      float o = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        S[e] = fmaf(k[8 * g + e], v[c], a.reverse ? S[e] : decay * S[e]);
        o = fmaf(q[8 * g + e], S[e], o);
        if (a.reverse) S[e] *= decay;
      }
      part[64 * g + c] = o;
    }
    __syncthreads();
    if (threadIdx.x < 64) {
      float o = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o += part[64 * e + c];
      o *= a.state_scale;
      if (c < d) at(a.out, t)[c] = __float2bfloat16_rn(o);
    }
  }
}

// 16 scores of a row in its own block times their decays, each difference by itself.
__device__ __noinline__ void steep_block(uint32_t (&x)[16], const ChunkGates& w, float out_scale, int row, int j0) {
  const float hi = w.hi[row], lo = w.lo[row];
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    const float d = (hi - w.hi[j0 + j]) + (lo - w.lo[j0 + j]);
    x[j] = __float_as_uint(__uint_as_float(x[j]) * (out_scale * exp2_fast(d)));
  }
}

// DH: channels the tensor core works on (32 or 64).  GRAD: what the gates' gradient needs is written too.
template <int DH, bool ONLY_STATE, bool GRAD>
__global__ void __launch_bounds__(kThreads, 1)
    gated_tc_scan(const __grid_constant__ ScanSet p, const __grid_constant__ TcMaps maps) {
  using L = Layout<ONLY_STATE>;
  constexpr int kStages = L::kStages, kGateRing = L::kGateRing;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  uint8_t* kp = smem + L::kKp;
  uint8_t* planes = smem + L::kS;
  auto* gates = reinterpret_cast<typename L::Gates*>(smem + L::kGates);
  const ChunkGates* chunk_gate_ring = reinterpret_cast<const ChunkGates*>(gates);   // score and output warps
  Control& ctl = *reinterpret_cast<Control*>(smem + L::kControl);
  Bars& bar = ctl.bars;
  volatile uint32_t* abortf = &ctl.abort;
  constexpr int kKTile = ONLY_STATE ? 0 : kTileBytes, kVTile = kKTile + kTileBytes;

  const Scan& a = p.scan[blockIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool reverse = a.reverse;
  int64_t id = blockIdx.x;
  const int64_t nspans = ONLY_STATE ? p.spans - 1 : p.spans;   // the span last in order adds to no other
  const int64_t span = id % nspans + (ONLY_STATE && reverse ? 1 : 0);
  const int64_t bh = id / nspans, b = bh / p.H, h = bh % p.H;
  const int64_t first = span * p.span_chunks;
  const int count = static_cast<int>(min(p.span_chunks, p.chunks - first));
  auto chunk_of = [&](int n) { return first + (reverse ? count - 1 - n : n); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar.full + s, 1);
      mbar_init(bar.freed + s, ONLY_STATE ? kStateWarps : kStateWarps + kOutWarps);
    }
    for (int s = 0; s < kGateRing; ++s) {
      mbar_init(bar.gates + s, 1);
      mbar_init(bar.gates_freed + s, ONLY_STATE ? kStateWarps : kStateWarps + kOutWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar.scores + s, 1);
      mbar_init(bar.p_ready + s, kScoreWarps);
      mbar_init(bar.k_ready + s, ONLY_STATE ? kStateWarps + kScoreWarps : kStateWarps);
    }
    mbar_init(&bar.state_read, 1);
    mbar_init(&bar.out_done, 1);
    mbar_init(&bar.out_read, kOutWarps);
    mbar_init(bar.half_done, 1);
    mbar_init(bar.half_done + 1, 1);
    mbar_init(bar.l_done, 1);
    mbar_init(bar.l_done + 1, 1);
    mbar_init(&bar.s_ready, kStateWarps);
    mbar_init(bar.fin, 1);
    mbar_init(bar.fin + 1, 1);
    ctl.abort = 0u;
    ctl.bad = 0u;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&ctl.tmem, kTmemColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  // The scan behind its spans' states starts on the SMs that form none; its first loads do not depend on
  // them.  [4, 4096, 12, 64] forward 57.1 us in turn, 54.9 so.  (Other launches of a call stay in turn: small grids
  // that start early crowd the few SMs that are idle then: gradients of the same shape 1.2 times as long.)
  if (ONLY_STATE && threadIdx.x == 0) grid_dep_launch();
  if (!ONLY_STATE && warp <= kIssuer) ptx::grid_dep_wait();

  if (warp >= kGates) {
    // ------------------------------------------------------------ gates: the two warps take the chunks in turn
    const int me = warp - kGates;
    Sum all = {0.0f, 0.0f};
    float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (me < count) g = load_gates(p, b, h, chunk_of(me), lane);
    if (!ONLY_STATE) ptx::grid_dep_wait();
#pragma unroll 1
    for (int n = me; n < count; n += 2) {
      if (n >= kGateRing && !gwarp_wait(bar.gates_freed + n % kGateRing, n / kGateRing - 1, abortf)) break;
      const float4 now = g;
      if (n + 2 < count) g = load_gates(p, b, h, chunk_of(n + 2), lane);
      all = add(all, chunk_gates<ONLY_STATE>(now, gates[n % kGateRing], a, lane,
                                             GRAD && a.sums ? a.sums + (bh * p.chunks + chunk_of(n)) * (2 * kTcChunk) : nullptr));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.gates + n % kGateRing);
    }
    if (ONLY_STATE && lane == 0) ctl.decay[me] = all;
  } else if (warp == kIssuer) {
    // ------------------------------------------------------------ scores and outputs: MMAs
    if (!ONLY_STATE) {
      const bool leader = elect_one();
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTcChunk, false, false);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, DH, false, true);
      const uint64_t stage0 = smem_desc(smem_u32(smem), 16, kSbo, 2);           // K-major: q, k
      const uint64_t v0 = smem_desc(smem_u32(smem + kVTile), kSbo, kSbo, 2);    // MN-major: v
      const uint64_t state0 = smem_desc(smem_u32(planes), kSbo, kSbo, 2);
      auto scores = [&](int n) {
        const uint64_t q = stage0 + (n % kStages) * (L::kStage >> 4), k = q + (kKTile >> 4);
        const uint32_t d = tmem + kScores + 128 * (n & 1);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < DH / 16; ++ks) mma_bf16(d, q + 2 * ks, k + 2 * ks, idesc_s, ks > 0);
          mma_commit(bar.scores + (n & 1));
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int n = -1; n < count; ++n) {
        const int s = (n + kStages) % kStages;
        // the scores' other buffer: P of the chunk before has been read
        if (n > 0 && !gwarp_wait(&bar.out_done, n - 1, abortf)) break;
        if (n + 1 < count) {
          if (!gwarp_wait(bar.full + (n + 1) % kStages, (n + 1) / kStages, abortf)) break;
          tc_fence_after();
          scores(n + 1);
        }
        if (n < 0) continue;
        if (!gwarp_wait(&bar.s_ready, n, abortf)) break;
        if (n > 0 && !gwarp_wait(&bar.out_read, n - 1, abortf)) break;
        tc_fence_after();
        const uint64_t q = stage0 + s * (L::kStage >> 4), v = v0 + s * (L::kStage >> 4);
        if (leader) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks)
              mma_bf16(tmem + kO1, q + 2 * ks, state0 + (t * kStatePlane + ks * 2 * kSbo) / 16, idesc_o, t + ks > 0);
          mma_commit(&bar.state_read);
        }
        __syncwarp();
        if (!gwarp_wait(bar.p_ready + (n & 1), n >> 1, abortf)) break;
        tc_fence_after();
        const uint32_t pt = tmem + kScores + 128 * (n & 1);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < kTcChunk / 16; ++ks)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              mma_bf16_ts(tmem + kO2, pt + 16 * ks + 8 * t, v + ks * 2 * kSbo / 16, idesc_o, ks + t > 0);
          mma_commit(&bar.out_done);
        }
        __syncwarp();
      }
      if (leader) {
        mma_commit(bar.fin);
        drain_wait_on(bar.fin, 0, &g_gated_error);
      }
      __syncwarp();
    }
  } else if (warp == kAdder) {
    // ------------------------------------------------------------ loads; what the state gains: MMAs
    // what another launch of the call, or another scan, reads again stays in L2 (gradients of [4, 4096, 12, 64] 158, 153 us)
    const uint64_t policy = ONLY_STATE || GRAD ? policy_evict_last() : policy_evict_first();
    int issued = 0;
    auto load = [&](int n) {
      const int s = n % kStages;
      if (elect_one()) {
        uint8_t* st = smem + s * L::kStage;
        const int32_t t = static_cast<int32_t>(chunk_of(n) * kTcChunk), hh = static_cast<int32_t>(h),
                      bb = static_cast<int32_t>(b);
        mbar_arrive_expect_tx(bar.full + s, L::kStage);
        if (!ONLY_STATE) tma_load_4d(st, &maps.q[blockIdx.y], bar.full + s, 0, hh, t, bb, policy);
        tma_load_4d(st + kKTile, &maps.k[blockIdx.y], bar.full + s, 0, hh, t, bb, policy);
        tma_load_4d(st + kVTile, &maps.v[blockIdx.y], bar.full + s, 0, hh, t, bb, policy);
      }
      __syncwarp();
      ++issued;
    };
#pragma unroll 1
    for (int n = 0; n < min(count, kStages); ++n) load(n);
    if (!ONLY_STATE) ptx::grid_dep_wait();
    const bool leader = elect_one();
    constexpr uint32_t idesc = idesc_bf16_f32(64, DH, true, true);
    const uint64_t v0 = smem_desc(smem_u32(smem + kVTile), kSbo, kSbo, 2), k0 = smem_desc(smem_u32(kp), kSbo, kSbo, 2);
    bool ok = true;
    for (int n = 0; ok && n < count; ++n) {
      const int s = n % kStages;
      if (!gwarp_wait(bar.full + s, n / kStages, abortf)) break;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (!gwarp_wait(bar.k_ready + half, n, abortf)) { ok = false; break; }
        tc_fence_after();
        const uint64_t k = k0 + half * (4 * 2 * kSbo / 16), v = v0 + s * (L::kStage >> 4) + half * (4 * 2 * kSbo / 16);
        const uint32_t l = tmem + kL + (ONLY_STATE ? 64 * (n & 1) : 0);   // the state alone: two accumulators
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int t = 0; t < 3; ++t)
              mma_bf16(l, k + (t * kPlane + ks * 2 * kSbo) / 16, v + ks * 2 * kSbo / 16, idesc, half + ks + t > 0);
          if (ONLY_STATE) mma_commit(bar.half_done + half);
          if (half) mma_commit(bar.l_done + (ONLY_STATE ? n & 1 : 0));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (ONLY_STATE) {
        // the next chunk into the stage of chunk n - 1, whose k was scaled before its products
        if (n > 0 && n + kStages - 1 < count) {
          if (!gwarp_wait(bar.l_done + ((n - 1) & 1), (n - 1) >> 1, abortf)) break;
          load(n + kStages - 1);
        }
        continue;
      }
      // chunk n + 2 into the stage of chunk n - 1, once that is done with
      if (n > 0 && n + kStages - 1 < count) {
        if (!gwarp_wait(bar.freed + (n - 1) % kStages, (n - 1) / kStages, abortf)) break;
        load(n + kStages - 1);
      }
    }
    if (leader) {
      mma_commit(bar.fin + 1);
      drain_wait_on(bar.fin + 1, 0, &g_gated_error);
      for (int n = max(0, issued - kStages); n < issued; ++n)   // every load must have landed before the CTA ends
        drain_wait_on(bar.full + n % kStages, static_cast<uint32_t>((n / kStages) & 1), &g_gated_error);
    }
    __syncwarp();
  } else if (!ONLY_STATE && warp < kScoreWarps) {
    // ------------------------------------------------------------ scores
    const int q = warp & 3, half = warp >> 2, row = 32 * q + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
    // P of a chunk: this warp's 32 rows, tokens 64 half .., 16 tokens a round, their two
    // terms (8 columns each) over their scores.  A row's factor e^{b_i - m} waits for the
    // outputs, except where the row's block is steep.
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
      const int s = n % kStages;
      if (!gwarp_wait(bar.full + s, n / kStages, abortf) || !gwarp_wait(bar.gates + n % kGateRing, n / kGateRing, abortf)) break;
      const ChunkGates& w = chunk_gate_ring[n % kGateRing];
      // rows of v that are not finite (this warp looks at 32 of them, half a row a lane)
      {
        const uint8_t* v = smem + s * L::kStage + kVTile;
        const __nv_bfloat162 zero = __floats2bfloat162_rn(0.0f, 0.0f);
        __nv_bfloat162 z = zero;   // zero as long as what it meets is finite
#pragma unroll
        for (int u = 0; u < DH / 16; ++u) {
          const uint4 x = *reinterpret_cast<const uint4*>(v + unit_at(row, DH / 16 * half + u));
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&y[e]), zero, z);
        }
        if (*reinterpret_cast<const uint32_t*>(&z) & 0x7FFF7FFFu) *reinterpret_cast<volatile uint32_t*>(&ctl.bad) = 1u;
      }
      const bool steep = w.steep >> q & 1;
      if (!gwarp_wait(bar.scores + (n & 1), n >> 1, abortf)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 4 * half; c < 4 * half + 4; ++c) {   // 16 tokens
        const int cb = c >> 1, j0 = 16 * c;
        const uint32_t at = lanes + kScores + 128 * (n & 1) + j0;
        uint32_t t0[8], t1[8];
        if (reverse ? cb < q : cb > q) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t0[i] = t1[i] = 0u;
        } else {
          uint32_t x[16];
          tmem_ld_x16(at, x);
          tmem_ld_wait();
          if (cb == q && steep) {
            uint32_t z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = x[i];
            steep_block(z, w, a.out_scale, row, j0);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = z[i];
          } else {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 f = *reinterpret_cast<const float4*>(w.col[q] + j0 + j);
              float y[4];
              apart(mul(two(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), two(f.x, f.y)), y[0], y[1]);
              apart(mul(two(__uint_as_float(x[j + 2]), __uint_as_float(x[j + 3])), two(f.z, f.w)), y[2], y[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[j + e] = __float_as_uint(y[e]);
            }
            if (steep) {
              const float rw = w.row[row];
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * rw);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t t[2];
            split<2>(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), t);
            t0[i] = t[0];
            t1[i] = t[1];
          }
          if (cb == q) {   // tokens the row does not see: their bits cleared, whatever they hold
            const int seen = reverse ? row - j0 : row - j0 + 1;   // forwards tokens below it, backwards those from it
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = min(max(seen - 2 * i, 0), 2);
              uint32_t keep = k == 2 ? 0xFFFFFFFFu : k == 1 ? 0xFFFFu : 0u;
              if (reverse) keep = ~keep;
              t0[i] &= keep;
              t1[i] &= keep;
            }
          }
        }
        tmem_st_x8(at, t0);
        tmem_st_x8(at + 8, t1);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.p_ready + (n & 1));
    }
  } else if (warp >= kFirstOut) {
    // ------------------------------------------------------------ outputs
    if (!ONLY_STATE) {
      const int q = warp & 3, half = (warp - kFirstOut) >> 2, row = 32 * q + lane;
      const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q) << 16);
      const int64_t slice = half;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + b * a.out.sb + h * a.out.sh;
      const __nv_bfloat16* dot = static_cast<const __nv_bfloat16*>(a.dot.data) + b * a.dot.sb + h * a.dot.sh;
      // Output rows of chunk n, columns 32 half ..: through this warp's 2 KB of the q tile
      // (32 rows of 64 bytes), which nothing reads any more, so that eight rows go out at once.
      auto staged = [&](uint8_t* base, int r, int u) {
        return reinterpret_cast<uint4*>(base + 64 * r + ((u ^ (r >> 1 & 3)) << 4));
      };
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        const int s = n % kStages, part_row = lane >> 2, part = lane & 3;
        const int64_t t0 = chunk_of(n) * kTcChunk + 32 * q;
        const int rows = static_cast<int>(min(p.N - t0, static_cast<int64_t>(32)));   // in the sequence
        const bool part_in = 32 * half + 8 * part < p.d;
        uint4 z[4];
        if (GRAD && a.dots && 32 * half < DH) {
          const __nv_bfloat16* x = dot + (t0 + part_row) * a.dot.sn + 32 * half + 8 * part;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            z[i] = part_in && part_row + 8 * i < rows ? *reinterpret_cast<const uint4*>(x + 8 * i * a.dot.sn)
                                                      : make_uint4(0u, 0u, 0u, 0u);
        }
        const ChunkGates& w = chunk_gate_ring[n % kGateRing];
        if (!gwarp_wait(&bar.out_done, n, abortf)) break;
        tc_fence_after();
        const bool steep = w.steep >> q & 1;
        // o = f2 (f1 O1 + O2)
        const float f1 = steep ? w.enter[q] * w.row[row] : w.enter[q], f2 = steep ? 1.0f : w.row[row];
        float sum = 0.0f;
        uint8_t* mine = smem + s * L::kStage + 4096 * q + 2048 * half;
        if (GRAD && a.dots && 32 * half < DH) {
#pragma unroll
          for (int i = 0; i < 4; ++i) *staged(mine, part_row + 8 * i, part) = z[i];
          __syncwarp();
        }
#pragma unroll 1
        for (int c = 32 * half; c < min(32 * half + 32, DH); c += 16) {
          uint32_t x[16], y[16];
          tmem_ld_x16(lanes + kO1 + c, x);
          tmem_ld_x16(lanes + kO2 + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2)
              apart(mul(two(f2, f2), fma(two(f1, f1), two(__uint_as_float(x[8 * u + e]), __uint_as_float(x[8 * u + e + 1])),
                                         two(__uint_as_float(y[8 * u + e]), __uint_as_float(y[8 * u + e + 1])))),
                    o[e], o[e + 1]);
            uint4* at = staged(mine, lane, (c & 31) / 8 + u);
            if (GRAD && a.dots) {
              const uint4 r = *at;
              const uint32_t zz[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                sum = fmaf(__uint_as_float(x[8 * u + 2 * e]), low(zz[e]), fmaf(__uint_as_float(x[8 * u + 2 * e + 1]), high(zz[e]), sum));
            }
            *at = make_uint4(pack(o[0], o[1]), pack(o[2], o[3]), pack(o[4], o[5]), pack(o[6], o[7]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.out_read);
        if (32 * half < DH) {
          __nv_bfloat16* to = out + (t0 + part_row) * a.out.sn + 32 * half + 8 * part;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (part_in && part_row + 8 * i < rows)
              *reinterpret_cast<uint4*>(to + 8 * i * a.out.sn) = *staged(mine, part_row + 8 * i, part);
          // The tile's next contents come by TMA, which these stores must be in front of: the barrier
          // below orders ordinary accesses alone.
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar.freed + s);
          mbar_arrive(bar.gates_freed + n % kGateRing);
        }
        if (GRAD && a.dots && lane < rows && 32 * half < DH) a.dots[(slice * p.BH + bh) * p.N + t0 + lane] = f2 * (f1 * sum);
      }
    }
  } else {
    // ------------------------------------------------------------ the state
    const bool carries = warp >= kScoreWarps;   // ONLY_STATE: the score warps help with k alone
    const int q = warp & 3, hf = (warp - kScoreWarps) >> 2;
    const int r0 = 16 * q + (lane >> 2), c0 = 32 * hf + 2 * (lane & 3);
    const bool holds = carries && 16 * q < DH && 32 * hf < DH;   // of the state
    float S[16];
    if constexpr (ONLY_STATE) {
#pragma unroll
      for (int i = 0; i < 16; ++i) S[i] = 0.0f;
    } else {
      entering(S, a, bh, span, p.spans, p.d, [&](int i, int& r, int& c) {
        r = r0 + 8 * ((i >> 1) & 1);
        c = c0 + 8 * (i >> 2) + (i & 1);
        return holds && r < p.d && c < p.d;
      });
    }
    auto publish = [&]() {
      if (holds) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t t[2];
            split<2>(S[4 * n + 2 * e], S[4 * n + 2 * e + 1], t);
            uint8_t* at = planes + unit_at(r0 + 8 * e, 4 * hf + n) + 4 * (lane & 3);
            *reinterpret_cast<uint32_t*>(at) = t[0];
            *reinterpret_cast<uint32_t*>(at + kStatePlane) = t[1];
          }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.s_ready);
    };
    // k's rows, kRows at once, eight channels a lane: scaled and split into the planes.
    constexpr int kLanes = DH / 8, kRows = 32 / kLanes, kGroups = kTcChunk / kRows;
    const int kr = lane / kLanes, ku = lane % kLanes;
    auto scale_rows = [&](const uint8_t* k, const float* addw, uint8_t* to, int g0, int g1) {
#pragma unroll 1
      for (int g = g0; g < g1; ++g) {
        const int token = kRows * g + kr, at = unit_at(token, ku);
        const uint4 x = *reinterpret_cast<const uint4*>(k + at);
        const float f = addw[token];
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
        uint32_t t[4][3];
#pragma unroll
        for (int e = 0; e < 4; ++e) split<3>(mul(two(low(y[e]), high(y[e])), two(f, f)), t[e]);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          *reinterpret_cast<uint4*>(to + i * kPlane + at) = make_uint4(t[0][i], t[1][i], t[2][i], t[3][i]);
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    // S <- e^B S + L of chunk n
    auto gain = [&](int n, uint32_t l_columns) {
      const float total = gates[n % kGateRing].total;
      tc_fence_after();
      if (holds) {
        uint32_t l[16];
        tmem_ld_16x32(tmem + (static_cast<uint32_t>(32 * q) << 16) + l_columns + 32 * hf, l);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i += 2)
          apart(fma(two(total, total), two(S[i], S[i + 1]), two(__uint_as_float(l[i]), __uint_as_float(l[i + 1]))), S[i],
                S[i + 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar.freed + n % kStages);
        mbar_arrive(bar.gates_freed + n % kGateRing);
      }
    };
    if constexpr (ONLY_STATE) {
      // 16 warps scale, a half of the planes as soon as the products of the chunk before have
      // read it; the gain of a chunk is taken while the next one's products run
      const int g0 = warp * kGroups / 32, g1 = (warp + 1) * kGroups / 32;   // of a half
      bool ok = true;
#pragma unroll 1
      for (int n = 0; ok && n <= count; ++n) {
        if (n < count) {
          const int s = n % kStages;
          if (!gwarp_wait(bar.full + s, n / kStages, abortf) || !gwarp_wait(bar.gates + n % kGateRing, n / kGateRing, abortf))
            break;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            if (n > 0 && !gwarp_wait(bar.half_done + half, n - 1, abortf)) { ok = false; break; }
            scale_rows(smem + s * L::kStage + kKTile, gates[n % kGateRing].addw, kp, g0 + half * kGroups / 2,
                       g1 + half * kGroups / 2);
            if (lane == 0) mbar_arrive(bar.k_ready + half);
          }
          if (!ok) break;
        }
        if (n > 0 && carries) {
          if (!gwarp_wait(bar.l_done + ((n - 1) & 1), (n - 1) >> 1, abortf)) break;
          gain(n - 1, kL + 64 * ((n - 1) & 1));
        }
      }
    } else {
      // The score warps of a scheduler with fewer blocks of scores to form leave it more rows:
      // sixteenths of a half chunk per warp 3 3 | 3 2 | 2 1 | 1 1.  (Two each: 10% slower.)
      const int load = reverse ? 3 - q : q;   // 0: lightest score work
      const int from16 = load == 0 ? 3 * hf : load == 1 ? 6 + 3 * hf : load == 2 ? 11 + 2 * hf : 14 + hf;
      const int many16 = load == 0 ? 3 : load == 1 ? 3 - hf : load == 2 ? 2 - hf : 1;
      const int g0 = from16 * kGroups / 32, g1 = (from16 + many16) * kGroups / 32;   // of a half
#pragma unroll 1
      for (int n = 0; n < count; ++n) {
        const int s = n % kStages;
        if (n > 0 && !gwarp_wait(&bar.state_read, n - 1, abortf)) break;
        publish();
        if (!gwarp_wait(bar.full + s, n / kStages, abortf) || !gwarp_wait(bar.gates + n % kGateRing, n / kGateRing, abortf))
          break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          scale_rows(smem + s * L::kStage + kKTile, gates[n % kGateRing].addw, kp, g0 + half * kGroups / 2, g1 + half * kGroups / 2);
          if (lane == 0) mbar_arrive(bar.k_ready + half);
        }
        if (GRAD && a.entries && holds) {   // as the threads hold it
          float4* to = reinterpret_cast<float4*>(a.entries) + (bh * p.chunks + chunk_of(n)) * (DH * DH / 4) +
                       (warp - kScoreWarps) * 128 + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) to[32 * i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
        if (!gwarp_wait(bar.l_done, n, abortf)) break;
        gain(n, kL);
      }
    }
    // A scan's last state goes out behind everything else (it may lie where the first one does, which
    // redo_span reads), from where the scaled k was.
    float* to = ONLY_STATE ? a.local + (bh * p.spans + span) * p.d * p.d : reinterpret_cast<float*>(kp);
    const int width = ONLY_STATE ? p.d : 64;
    if (holds) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = r0 + 8 * ((i >> 1) & 1), c = c0 + 8 * (i >> 2) + (i & 1);
        if (r < p.d && c < p.d) to[r * width + c] = S[i];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemColumns);
  if (ONLY_STATE && threadIdx.x == 0)
    a.decay[bh * p.spans + span] = exp2_of(add(ctl.decay[0], ctl.decay[1]), Sum{0.0f, 0.0f});
  if (!ONLY_STATE && *reinterpret_cast<volatile uint32_t*>(&ctl.bad) && !ctl.abort)
    redo_span(p, a, smem, bh, span, first * kTcChunk, min(p.N, (first + count) * kTcChunk));
  if (!ONLY_STATE && a.last && span == (reverse ? 0 : p.spans - 1)) {
    const float* from = reinterpret_cast<const float*>(kp);
    for (int i = threadIdx.x; i < p.d * p.d; i += kThreads)
      a.last[bh * p.d * p.d + i] = from[i / p.d * 64 + i % p.d];
  }
}

bool operand_map(const ScanSet& set, int64_t B, const Operand& o, CUtensorMap* m) {
  const int64_t lim = int64_t{1} << 39;   // strides in bytes below 2^40
  const int64_t sh = set.H > 1 ? o.sh : set.d, sn = set.N > 1 ? o.sn : set.d, sb = B > 1 ? o.sb : set.d;
  if (sh <= 0 || sn <= 0 || sb <= 0 || sh >= lim || sn >= lim || sb >= lim) return false;   // a shared row: no map
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(set.d), static_cast<cuuint64_t>(set.H),
                              static_cast<cuuint64_t>(set.N), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(sh * 2), static_cast<cuuint64_t>(sn * 2),
                                 static_cast<cuuint64_t>(sb * 2)};
  const cuuint32_t box[4] = {64u, 1u, static_cast<cuuint32_t>(kTcChunk), 1u};
  return encode_tensor_map(m, 4, o.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int DH, bool ONLY_STATE, bool GRAD = false>
int launch(const ScanSet& set, const TcMaps& maps, int scans, cudaStream_t s) {
  constexpr int kBytes = static_cast<int>(Layout<ONLY_STATE>::kBytes);
  // a per-device setting: made on every call, for whichever device is current
  if (cudaFuncSetAttribute(gated_tc_scan<DH, ONLY_STATE, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) !=
      cudaSuccess)
    return MHLA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(set.BH * (ONLY_STATE ? set.spans - 1 : set.spans));
  KernelTimer timer(ONLY_STATE ? "gated_tc_span_state" : "gated_tc_scan", s);
  if (!ONLY_STATE && set.scan[0].join)   // directly behind the states of the spans
    return launch_dependent(gated_tc_scan<DH, ONLY_STATE, GRAD>, dim3(grid, scans), dim3(kThreads), kBytes, s, set, maps) ==
                   cudaSuccess
               ? MHLA_OK
               : MHLA_ERR_CUDA;
  gated_tc_scan<DH, ONLY_STATE, GRAD><<<dim3(grid, scans), kThreads, kBytes, s>>>(set, maps);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

}  // namespace

bool tc_supported(const GatedProblem& p) {
  return p.dtype == MHLA_BF16 && p.d <= 64 && p.d % 8 == 0 && p.N < (int64_t{1} << 31) - kTcChunk;
}

// One CTA an SM: as many spans as fill the SMs once, none shorter than two chunks; up to four
// chunks stay whole (a chunk takes 2.6 us; a second span's launch and start more than two of them).
Cut tc_cut(const GatedProblem& p, int scans) {
  Cut c;
  c.chunks = (p.N + kTcChunk - 1) / kTcChunk;
  const int64_t spans = std::max<int64_t>(1, kSms / (p.B * p.H * scans));
  c.span_chunks = c.chunks <= 4 ? c.chunks : std::max<int64_t>(2, (c.chunks + spans - 1) / spans);
  c.spans = (c.chunks + c.span_chunks - 1) / c.span_chunks;
  return c;
}

bool tc_maps(const GatedProblem& p, const ScanSet& set, int scans, TcMaps* maps) {
  ScanSet sizes = {};
  sizes.N = p.N; sizes.H = p.H; sizes.d = p.d;
  for (int i = 0; i < scans; ++i)
    if (!operand_map(sizes, p.B, set.scan[i].q, &maps->q[i]) || !operand_map(sizes, p.B, set.scan[i].k, &maps->k[i]) ||
        !operand_map(sizes, p.B, set.scan[i].v, &maps->v[i]))
      return false;
  return true;
}

int launch_tc_scan(const ScanSet& set, const TcMaps& maps, int scans, bool span_state, cudaStream_t s) {
  const bool narrow = set.d <= 32;
  if (span_state) return narrow ? launch<32, true>(set, maps, scans, s) : launch<64, true>(set, maps, scans, s);
  if (scans > 1) return narrow ? launch<32, false, true>(set, maps, scans, s) : launch<64, false, true>(set, maps, scans, s);
  return narrow ? launch<32, false>(set, maps, scans, s) : launch<64, false>(set, maps, scans, s);
}

}  // namespace gated

int read_and_clear_gated_error(void* stream, uint32_t* flags) { return tc::read_and_clear_word(g_gated_error, stream, flags); }

MHLA_DEFINE_STALL_SETTER(set_stall_gated)

}  // namespace mhla
