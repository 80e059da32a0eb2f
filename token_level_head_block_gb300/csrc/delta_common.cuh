// What the kernels of the gated delta rule share: sizes, the layout of what one kernel leaves for the
// next in the workspace, and fragments.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gated_common.cuh"
#include "mhla_internal.h"
#include "ptx.cuh"
#include "stall_hook.cuh"
#include "warp_mma.cuh"

namespace mhla {
namespace delta {

using namespace gated;

// How values enter the tensor cores.
//
// The chain, from chunk to chunk, takes fp16 at a scale: a block's largest value is brought to [2^14, 2^15) by a power of two, near
// fp16's end, so that its last bit, 2^-24, lies as far below as it can; sums of 128 products of two such values stay below 2^37.
// A value is then one fp16 (2^-11 of it, or 2^-39 of the largest), or two (2^-22, 2^-39).  Brought to [1, 2) a token's value of 1e-6 of a
// later one's in its block was 2% off, which a causal result may not be.  What reaches the float32 state
// (the state, w, K^) takes two; bf16 inputs are exact in one but for that 2^-39; what only feeds bf16 outputs takes one.  Three products
// of two such terms stand for six of three bf16 ones, and the chain's time is its products.  A scale belongs to 16 columns of
// a row of the state, of w or of e^{B-b} w, to 16 rows of K^, to a row of Q or the scores, to a chunk of K.
//
// In delta_prepare, and in what delta_back forms ahead, values are sums of bf16 terms, which need no scale: an input one (bf16) or three
// (float32), a value that reaches the state three (2^-24).  delta_grads takes every plane of a chunk as fp16 at one scale,
// but dout and A in dq's products, whose rows stand for a token's own gradient, at a row's.
// Tokens a chunk: three planes of float32 rows of 128 channels leave room for 32.
template <typename T>
struct Form;
template <>
struct Form<__nv_bfloat16> {
  static constexpr int kIn = 1, kHalves = 1, kChunk = 64;
};
template <>
struct Form<float> {
  static constexpr int kIn = 3, kHalves = 2, kChunk = 32;
};
constexpr int kChain = 3;   // bf16 terms on the way to the state

// A chunk's values a token, then whether any is not finite and each column's first such token.
template <int C, int DK>
struct Marks {
  float douts[C];          // gradients: the scale of dout's row
  float hi[C], lo[C];      // sum b of the log decays up to the token, in powers of two
  float inside[C];         // e^b
  float query[C];          // scale e^b and the scale of Q's row
  float score[C];          // the scale of the scores' row
  float after[C];          // e^(B - b), B that of the whole chunk
  float beta[C];
  float keys[4];           // the scale of each 16 rows of K^
  float total;             // e^B
  float key;               // the scale of K
  int32_t any;
  float inverse, queries, pad[3];   // gradients: the scales of T and Q
  int32_t first[DK];
};

// One 16 x 16 block of an operand as the 32 lanes hold it, 16 bytes a lane.  What one kernel forms the next takes block by
// block, each lane its own bytes, with no shuffling in between.
constexpr int kBlock = 512;

template <typename T, int DK>
struct Lay {
  static constexpr int C = Form<T>::kChunk, kIn = Form<T>::kIn, kHalves = Form<T>::kHalves;
  static constexpr int kTiles = C / 16, kSides = DK / 16;          // blocks of a chunk's tokens, of the channels
  static constexpr bool kApart = kIn > 1;
  static constexpr int kRows = C * DK * 2, kSquare = C * C * 2;   // bytes of a plane
  static constexpr int kInput = kIn * kRows, kInputHalf = kHalves * kRows, kKeys = 2 * kRows, kInverse = kHalves * kSquare;
  static constexpr int kScores = kHalves * kSquare, kScoresBack = kChain * kSquare;
  static constexpr int kTokens = C / 8 * kBlock, kState = DK / 8 * kBlock;   // of 16 columns, float32 fragments
  using M = Marks<C, DK>;
  static constexpr int kMarks = sizeof(M);
  static_assert(kMarks % 16 == 0, "copied in 16-byte units");
};

// Where a call's images lie, of every chunk [B][Hk][chunks] (inputs of key heads) or [B][H][chunks].  Blocks of an operand with
// its terms side by side; k runs fastest, after the terms.  tok: blocks of tokens, ch: of channels; fp16 but for q_add,
// scores_back and dout_cols.
struct Images {
  char* k_add;          // K as [k = tok][n = ch], blocks [ch][tok]
  char* q_rows;         // Q as [m = tok][k = ch], blocks [tok][ch]
  char* keys;           // T beta e^b K as [n = tok][k = ch], blocks [tok][ch]
  char* scores;         // scale tril(Q K^T . decay) as [m = tok][k = tok], blocks [tok][tok]
  char* u;              // (T beta V)^T, float32 fragments [ch][C / 8][32]
  char* marks;
  // gradients
  char *k, *q, *dout, *inverse;   // planes of rows at a scale each; T
  char* k_rows;         // K as [n = tok][k = ch], blocks [tok][ch]
  char* keys_add;       // T beta e^b K as [k = tok][n = ch], blocks [ch][tok]
  char* q_add;          // Q as [k = tok][n = ch], blocks [ch][tok]
  char* scores_back;    // the scores as [k = tok][n = tok], blocks [n][k]
  char* dout_cols;      // dout^T as [m = ch][k = tok], blocks [ch][tok]
  char *s, *w;          // the state entering the chunk and what its tokens write, float32 fragments
  char *ds, *dw;        // gradients: of the state leaving the chunk and of w
};

struct Common {
  Operand q, k, v, g, beta, dout;
  int64_t N, H, Hk;
  uint32_t chunks;
  int32_t d;
  float scale;
  uint32_t wide;        // operands whose rows 16-byte accesses take, a bit each in the order above
  Images im;
};
enum : uint32_t { kWideQ = 1, kWideK = 2, kWideV = 4, kWideDout = 8 };

// fp16 at a scale: the power of two that brings `most` to [2^14, 2^15), and what undoes it; both are normal.
struct Scale {
  float to, from;
};
__device__ __forceinline__ Scale scale_of(float most) {
  constexpr uint32_t kUp = 14;
  const uint32_t e = min(max(__float_as_uint(most) >> 23, kUp + 1), 254u);
  return Scale{__uint_as_float((254u + kUp - e) << 23), __uint_as_float((e - kUp) << 23)};
}
// The scale of a whole plane of a chunk, from the bits of its largest; with an infinity in it all of it becomes NaN, not zero.
__device__ __forceinline__ Scale plane_scale(uint32_t most) {
  const Scale by = scale_of(__uint_as_float(most));
  return most < 0x7F800000u ? by : Scale{__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u)};
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// A pair as one fp16 each or the sum of two.
template <int NT>
__device__ __forceinline__ void halves(float x, float y, uint32_t (&t)[NT]) {
  t[0] = pack_half(x, y);
  if constexpr (NT > 1) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&t[0]));
    t[1] = pack_half(x - f.x, y - f.y);
  }
}
// c = sum over the pairs of terms that matter, small ones first; each tile begins anew.  step 0 .. steps - 1 of it.
template <int NA, int NB>
__device__ __forceinline__ constexpr int product_steps() { return 1 + (NA > 1) + (NB > 1); }
template <int NA, int NB>
__device__ __forceinline__ void product(float (&c)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4], int half, int step) {
  const int last = product_steps<NA, NB>() - 1;
  const int i = NA > 1 && step == 0 ? 1 : 0, j = NB > 1 && step == last - 1 ? 1 : 0;
  if (step == 0)
    mma_half_first(c, a[i < NA ? i : 0], b[j < NB ? j : 0][2 * half], b[j < NB ? j : 0][2 * half + 1]);
  else
    mma_half(c, a[i < NA ? i : 0], b[j < NB ? j : 0][2 * half], b[j < NB ? j : 0][2 * half + 1]);
}
template <int NA, int NB>
__device__ __forceinline__ void products(float (&c)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4], int half) {
#pragma unroll
  for (int step = 0; step < product_steps<NA, NB>(); ++step) product(c, a, b, half, step);
}
// Two steps of 16 of k of MT x NT tiles, NP of a[k][m] and b[k][n / 2]; the k-th step's sum is added at its rows' scale.  The MMAs of one
// tile lie 2 MT NT apart, so none waits for the one before.
template <int MT, int NT, int NA, int NB, typename ScaleOf>
__device__ __forceinline__ void add_scaled(float (&sum)[MT][NT][4], const uint32_t (&a)[2][MT][NA][4], const uint32_t (&b)[2][NT / 2][NB][4],
                                           ScaleOf scale) {
  float c[2][MT][NT][4];
#pragma unroll
  for (int step = 0; step < product_steps<NA, NB>(); ++step)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) product(c[k][m][n], a[k][m], b[k][n >> 1], n & 1, step);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const float2 f = scale(k, m);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sum[m][n][0] = fmaf(c[k][m][n][0], f.x, sum[m][n][0]); sum[m][n][1] = fmaf(c[k][m][n][1], f.x, sum[m][n][1]);
        sum[m][n][2] = fmaf(c[k][m][n][2], f.y, sum[m][n][2]); sum[m][n][3] = fmaf(c[k][m][n][3], f.y, sum[m][n][3]);
      }
    }
}
// The same, added to c.
template <int NA, int NB>
__device__ __forceinline__ void add_products(float (&c)[4], const uint32_t (&a)[NA][4], const uint32_t (&b)[NB][4], int half) {
  if constexpr (NA > 1) mma_half(c, a[1], b[0][2 * half], b[0][2 * half + 1]);
  if constexpr (NB > 1) mma_half(c, a[0], b[1][2 * half], b[1][2 * half + 1]);
  mma_half(c, a[0], b[0][2 * half], b[0][2 * half + 1]);
}
// The largest size among the four lanes of a row.
__device__ __forceinline__ float over_row(float m) {
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  return fmaxf(m, __shfl_xor_sync(~0u, m, 2));
}

struct ScanArgs {
  Common c;
  const float* init;
  float* last;
  Operand out;
  bool out_pairs;       // 4-byte stores of two bf16 (8-byte of two float32) take the output
};

__device__ __forceinline__ float nan_value() { return __int_as_float(0x7FFFFFFF); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7F800000); }

// float32 fragments of a transposed product [m][n] as A operands: 16 of k from column tiles 2 ks, 2 ks + 1.
template <int NT>
__device__ __forceinline__ void as_rows(uint32_t (&a)[NT][4], const float (&lo)[4], const float (&hi)[4]) {
  uint32_t t[NT];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float(&x)[4] = e < 2 ? lo : hi;
    split<NT>(x[2 * (e & 1)], x[2 * (e & 1) + 1], t);
#pragma unroll
    for (int i = 0; i < NT; ++i) a[i][e] = t[i];
  }
}

__device__ __forceinline__ void copy_async(uint32_t dst, const char* src, int bytes, int thread, int threads) {
  for (int i = 16 * thread; i < bytes; i += 16 * threads) cp_async_16(dst + i, src + i, 16);
}
__device__ __forceinline__ void load_block(uint32_t (&r)[4], const char* smem, int block, int lane) {
  const uint4 x = *reinterpret_cast<const uint4*>(smem + block * kBlock + 16 * lane);
  r[0] = x.x; r[1] = x.y; r[2] = x.z; r[3] = x.w;
}
// The transpose of an 8 x 8 tile, a pair of its row a lane.
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Waits for a phase of a barrier that copies complete on.  Bounded: one that gives up is reported in *error and false for the
// whole warp, which then waits (again for so long at most) for the copies that are still in flight and asks for no more.
static __device__ __noinline__ bool wait_copies_long(uint64_t* bar, uint32_t parity, unsigned int* error) {
  if (stall_this_warp()) {   // a test's: it gives up, and the copies in flight are waited for behind it
    volatile uint32_t none = 0;
    stalled_wait(&none);
    atomicOr(error, 1u);
  }
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t it = 1; it < (1u << 28); ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0 && ptx::globaltimer() - t0 > 2000000000ull) break;
  }
  atomicOr(error, 1u);
  return false;
}
__device__ __forceinline__ bool wait_copies(uint64_t* bar, uint32_t parity, unsigned int* error) {
  return __all_sync(~0u, ptx::mbar_try_wait(bar, parity) || wait_copies_long(bar, parity, error));
}

template <typename T>
__device__ __forceinline__ void store_pair(T* p, float x, float y, bool pairs, bool both);
template <>
__device__ __forceinline__ void store_pair<__nv_bfloat16>(__nv_bfloat16* p, float x, float y, bool pairs, bool both) {
  if (pairs) {
    *reinterpret_cast<uint32_t*>(p) = pack(x, y);
  } else {
    from_f(p, x);
    if (both) from_f(p + 1, y);
  }
}
template <>
__device__ __forceinline__ void store_pair<float>(float* p, float x, float y, bool pairs, bool both) {
  if (pairs) {
    *reinterpret_cast<float2*>(p) = make_float2(x, y);
  } else {
    p[0] = x;
    if (both) p[1] = y;
  }
}

inline int padded(int d) { return d <= 32 ? 32 : d <= 64 ? 64 : 128; }

// Launches of delta_forward.cu that both directions make.
int launch_prepare(const Common& c, int64_t BH, int dtype, bool grad, cudaStream_t s);
int launch_scan(const ScanArgs& a, int64_t BH, int dtype, bool keep, cudaStream_t s);
size_t lay_out(const DeltaProblem& p, bool grad, char* base, Images* im);
Common common(const DeltaProblem& p, const Operand* dout);
// Whether a chain's CTA takes 32 columns of the state (heads of 33 to 64 channels) or 16, as the others always do.
bool two_tiles(int64_t BH, int d, int64_t most);
bool pairs_fit(const Operand& o, int d, int dtype);

}  // namespace delta
}  // namespace mhla
