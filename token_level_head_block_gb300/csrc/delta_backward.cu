// Gradients of the gated delta rule (delta_forward.cu has the notation).  With S the state that enters a chunk, D the gradient
// of the one that leaves it, P = scale tril(Q K^T . D_ij) and do the gradient of the outputs,
//   dW = P^T do + (e^{B-b} K) D          dR = T^T dW
//   D' = e^B D + (scale e^b Q)^T do - K^^T dW      of the state that enters
// so the gradient of the state runs backwards through a chunk in two products, as the state itself runs forwards: delta_back is
// delta_scan's chain turned round, the warps beside it a chunk ahead with P^T do and Q^T do.  What is left,
//   A = scale (do W^T) . D_ij  (i >= j),   L = -beta (dR W^T) . D_ij  (i > j)
//   dq = scale e^b do S^T + A K
//   dk = A^T Q + L K + L^T K - beta e^b dR S^T + e^{B-b} W D^T
//   dv = beta dR,   dbeta = dR . (V - e^b K S) - rows of (dR W^T . G)
// and the gates', a sum over what has the gate between its two tokens (pairs A (q k) + L (k k), what reads the state behind
// it, what writes D in front of it, and e^B <S, D>; nothing cancels), every chunk does by itself: delta_grads.
//
// Measured, bf16 [4, 4096, 12, 64]:
//   delta_prepare 131 us, delta_states (delta_scan with its states and W kept) 74
//   delta_back    126 us, 2.0 us a chunk: the chain's two products, which share an SM's issue slots with the warps beside it; one such warp
//                 for two took 142
//   delta_grads   213 us: 160 KB read and written a chunk (75 us of HBM's time), 40,000 cycles a chunk, two of them on an SM at once, of which
//                 10,000 wait for what it reads.  Values and their gradients element by element from memory took 315 us, sums of bf16
//                 terms for fp16 351; the images of the CTA that follows asked for as far as L2 220.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "delta_common.cuh"
#include "tc_common.cuh"

namespace mhla {

__device__ unsigned int g_delta_back_error = 0;

using namespace delta;

namespace {

struct BackArgs {
  Common c;
  const float* last;    // gradient of the last state, or null for zero
  float* first;         // of the first one, or null
};

// A CTA walks the chunks backwards with 16 MT columns of the state's gradient, as delta_scan does forwards; the warps beside the
// chain's fetch what both read and form, a chunk ahead, what of it does not wait for the chain.
template <typename T, int DK, int MT>
struct BackLay {
  using L = Lay<T, DK>;
  using M = typename L::M;
  static constexpr int kWarps = L::kTiles, kThreads = 96 * kWarps;   // the chain's; with those beside it
  static constexpr int kShare = DK / 16 < kWarps ? 1 : DK / 16 / kWarps;   // blocks of the state's rows a warp
  static constexpr int kHand = MT * (2 + 2 * kShare) * kBlock;           // a warp's part of P^T do and Q^T do
  static constexpr int kStatePlane = 16 * MT * DK * 2, kTokenPlane = 16 * MT * L::C * 2;
  static constexpr int kState = 0, kW = kState + 2 * kStatePlane, kStateScale = kW + 2 * kTokenPlane;
  static constexpr int kTokenScale = kStateScale + 16 * MT * L::kSides * 4, kHands = (kTokenScale + 16 * MT * L::kTiles * 4 + 127) / 128 * 128;
  static constexpr int kRing = kHands + 2 * kWarps * kHand;
  // of a chunk, the chain's: blocks of K, of K^
  static constexpr int kKBytes = L::kSides * L::kHalves * kBlock, kKeysBytes = kShare * L::kTiles * 2 * kBlock;
  static constexpr int kKeys = kKBytes, kPair = kKeys + kKeysBytes;
  static constexpr int kMarkFrom = offsetof(M, after), kMarkBytes = offsetof(M, first) - kMarkFrom;
  static constexpr int kMarks = kWarps * kPair, kStage = kMarks + (kMarkBytes + 127) / 128 * 128;
  // and of the next chunk, what is formed ahead: of dout, of the scores, of Q, e^b
  static constexpr int kDoutBytes = MT * L::kTiles * L::kIn * kBlock, kScoreBytes = L::kTiles * kChain * kBlock;
  static constexpr int kQBytes = kShare * L::kTiles * L::kIn * kBlock, kInsideBytes = L::C * 4;
  static constexpr int kScores = kDoutBytes, kFirst = kScores + kScoreBytes;                             // a warp that forms P^T do
  static constexpr int kQ = kDoutBytes, kInside = kQ + kQBytes, kSecond = kInside + kInsideBytes;        // and one that forms Q^T do
  static constexpr int kFirsts = kRing + 2 * kStage, kSeconds = kFirsts + kWarps * kFirst;
  static constexpr int kBytes = kSeconds + kWarps * kSecond;
  static_assert(kBytes <= 226 * 1024, "shared memory");
  static_assert(kMarkFrom % 16 == 0 && kMarkBytes % 16 == 0 && kPair % 128 == 0 && kFirst % 128 == 0 && kSecond % 128 == 0, "copied in units of 16 bytes");
};

template <typename T, int DK, int MT>
__global__ void __launch_bounds__(BackLay<T, DK, MT>::kThreads) delta_back(const __grid_constant__ BackArgs a) {
  using W = BackLay<T, DK, MT>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, TILES = L::kTiles, SIDES = L::kSides, SHARE = W::kShare;
  extern __shared__ __align__(128) char smem[];
  __shared__ uint64_t bars[TILES][4];   // of either stage of the chain's operands, of what either warp beside it forms ahead
  const Common& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (p.d + 16 * MT - 1) / (16 * MT);
  const int64_t bh = blockIdx.x / groups, b = bh / p.H, h = bh % p.H, key = b * p.Hk + h / (p.H / p.Hk);
  const int tile0 = static_cast<int>(blockIdx.x % groups) * MT;
  const uint32_t base = ptx::smem_u32(smem);
  const int count = static_cast<int>(p.chunks);
  const int own = warp % TILES;
  const int g = lane >> 2, t = 2 * (lane & 3);
  const bool shares = own * SHARE < SIDES;   // a warp of the chain has rows of the state
  auto sync = [&]() { ptx::named_bar_sync(1, W::kThreads); };   // of the CTA, from several places in the code
  auto chunk_of = [&](int i) { return bh * p.chunks + (count - 1 - i); };
  auto key_chunk_of = [&](int i) { return key * p.chunks + (count - 1 - i); };

  // The warps beside the chain: the first of 16 tokens (a share of the state's rows) fetches for the chain and forms (P^T do)^T, the
  // second ((scale e^b Q)^T do)^T.
  if (warp >= TILES) {
    const bool first = warp < 2 * TILES;
    uint64_t *bar = bars[own], *bar_ahead = bar + (first ? 2 : 3);
    if (lane == 0) {
      if (first) {
        ptx::mbar_init(bar, 1);
        ptx::mbar_init(bar + 1, 1);
      }
      ptx::mbar_init(bar_ahead, 1);
      ptx::fence_mbar_init();
    }
    __syncwarp();
    bool alive = first || shares;   // and no wait has given up
    char* const st = smem + (first ? W::kFirsts + own * W::kFirst : W::kSeconds + own * W::kSecond);
    auto load = [&](int i) {   // the chain's
      if (!first || lane != 0 || i >= count || !alive) return;
      char* stage = smem + W::kRing + (i & 1) * W::kStage;
      char* to = stage + own * W::kPair;
      uint64_t* on = bar + (i & 1);
      ptx::mbar_arrive_expect_tx(on, W::kKBytes + (shares ? W::kKeysBytes : 0) + (own == 0 ? W::kMarkBytes : 0));
      ptx::bulk_load_plain(to, p.im.k_rows + key_chunk_of(i) * L::kInputHalf + own * W::kKBytes, W::kKBytes, on);
      if (shares) ptx::bulk_load_plain(to + W::kKeys, p.im.keys_add + chunk_of(i) * L::kKeys + own * W::kKeysBytes, W::kKeysBytes, on);
      if (own == 0) ptx::bulk_load_plain(stage + W::kMarks, p.im.marks + chunk_of(i) * L::kMarks + W::kMarkFrom, W::kMarkBytes, on);
    };
    const uint32_t seen = (TILES - own) * kChain * kBlock;   // scores from the diagonal on
    auto load_ahead = [&](int i) {
      if (lane != 0 || i >= count || !alive) return;
      ptx::mbar_arrive_expect_tx(bar_ahead, W::kDoutBytes + (first ? seen : W::kQBytes + W::kInsideBytes));
      ptx::bulk_load_plain(st, p.im.dout_cols + chunk_of(i) * L::kInput + tile0 * TILES * L::kIn * kBlock, W::kDoutBytes, bar_ahead);
      if (first) {
        ptx::bulk_load_plain(st + W::kScores + own * kChain * kBlock,
                             p.im.scores_back + chunk_of(i) * L::kScoresBack + own * (TILES + 1) * kChain * kBlock, seen, bar_ahead);
        return;
      }
      ptx::bulk_load_plain(st + W::kQ, p.im.q_add + key_chunk_of(i) * L::kInput + own * W::kQBytes, W::kQBytes, bar_ahead);
      ptx::bulk_load_plain(st + W::kInside, p.im.marks + chunk_of(i) * L::kMarks + offsetof(typename L::M, inside), W::kInsideBytes, bar_ahead);
    };
    auto ahead = [&](int i) {
      float4* hand = reinterpret_cast<float4*>(smem + W::kHands + ((i & 1) * TILES + own) * W::kHand) + lane;
      if (first) {
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          Accumulators<2, true> y;
          y.clear();
#pragma unroll
          for (int ks = 0; ks < TILES; ++ks) {
            if (ks < own) continue;
            uint32_t o[L::kIn][4], s[kChain][1][4];
#pragma unroll
            for (int k = 0; k < L::kIn; ++k) load_block(o[k], st, (n * TILES + ks) * L::kIn + k, lane);
#pragma unroll
            for (int k = 0; k < kChain; ++k) load_block(s[k][0], st + W::kScores, ks * kChain + k, lane);
            mma_terms(y, 0, o, s);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            hand[32 * (n * (2 + 2 * SHARE) + j)] = make_float4(y.get(j, 0), y.get(j, 1), y.get(j, 2), y.get(j, 3));
        }
        return;
      }
      if (!shares) return;
      const float* inside = reinterpret_cast<const float*>(st + W::kInside);
#pragma unroll
      for (int n = 0; n < MT; ++n) {
        Accumulators<2 * SHARE, true> x;
        x.clear();
#pragma unroll
        for (int ks = 0; ks < TILES; ++ks) {
          float f[4][2];
#pragma unroll
          for (int k = 0; k < L::kIn; ++k) {
            uint32_t o[4];
            load_block(o, st, (n * TILES + ks) * L::kIn + k, lane);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e][0] = k == 0 ? low(o[e]) : f[e][0] + low(o[e]);
              f[e][1] = k == 0 ? high(o[e]) : f[e][1] + high(o[e]);
            }
          }
          uint32_t oa[kChain][4], q[L::kIn][SHARE][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 in = *reinterpret_cast<const float2*>(inside + 16 * ks + 8 * (e >> 1) + t);
            uint32_t z[kChain];
            split<kChain>(f[e][0] * (p.scale * in.x), f[e][1] * (p.scale * in.y), z);
#pragma unroll
            for (int k = 0; k < kChain; ++k) oa[k][e] = z[k];
          }
#pragma unroll
          for (int k = 0; k < L::kIn; ++k)
#pragma unroll
            for (int j = 0; j < SHARE; ++j) load_block(q[k][j], st + W::kQ, (j * TILES + ks) * L::kIn + k, lane);
          mma_terms(x, 0, oa, q);
        }
#pragma unroll
        for (int j = 0; j < 2 * SHARE; ++j)
          hand[32 * (n * (2 + 2 * SHARE) + 2 + j)] = make_float4(x.get(j, 0), x.get(j, 1), x.get(j, 2), x.get(j, 3));
      }
    };
    load_ahead(0);
    load(0);
    if (alive && stall_this_warp()) wait_copies_long(bar_ahead, 0, &g_delta_back_error);   // a test's
    // the chain's copies of chunk i and, ahead, those of chunk j: waited for once more when a wait has given up
    auto give_up = [&](int i, int j) {
      alive = false;
      if (first && i < count) wait_copies_long(bar + (i & 1), i >> 1 & 1, &g_delta_back_error);
      if (j < count) wait_copies_long(bar_ahead, j & 1, &g_delta_back_error);
    };
    if (alive && !wait_copies(bar_ahead, 0, &g_delta_back_error)) give_up(0, 0);
    ahead(0);
    __syncwarp();
    load_ahead(1);
    for (int i = 0; i < count; ++i) {
      if (first && alive && !wait_copies(bar + (i & 1), i >> 1 & 1, &g_delta_back_error)) give_up(i, i + 1);
      sync();   // the chunk's operands, what was formed ahead and the planes of D are there; the chunk before is done with
      load(i + 1);
      if (i + 1 < count) {
        if (alive && !wait_copies(bar_ahead, i + 1 & 1, &g_delta_back_error)) give_up(i + 1, i + 1);
        ahead(i + 1);
        __syncwarp();
        load_ahead(i + 2);
      }
      sync();
    }
    return;
  }

  // D^T as delta_scan holds S^T
  float D[MT][2 * SHARE][4];
  auto publish = [&]() {
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < SHARE; ++j)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const float x[4] = {D[n][2 * j][2 * f], D[n][2 * j][2 * f + 1], D[n][2 * j + 1][2 * f], D[n][2 * j + 1][2 * f + 1]};
          const Scale by = scale_of(over_row(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])))));
          const int row = 16 * n + g + 8 * f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t h[2];
            halves<2>(x[2 * e] * by.to, x[2 * e + 1] * by.to, h);
            char* to = smem + W::kState + unit_at<DK>(row, 2 * (own * SHARE + j) + e) + 2 * t;
            *reinterpret_cast<uint32_t*>(to) = h[0];
            *reinterpret_cast<uint32_t*>(to + W::kStatePlane) = h[1];
          }
          if ((lane & 3) == 0) reinterpret_cast<float*>(smem + W::kStateScale)[row * SIDES + own * SHARE + j] = by.from;
        }
  };
  if (shares) {
    const float* in = a.last ? a.last + bh * p.d * p.d : nullptr;
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * own * SHARE + 8 * j + t + (e & 1), c = 16 * (tile0 + n) + g + 8 * (e >> 1);
          D[n][j][e] = in && r < p.d && c < p.d ? in[static_cast<int64_t>(r) * p.d + c] : 0.0f;
        }
    publish();
  }
  for (int i = 0; i < count; ++i) {
    const char* stage = smem + W::kRing + (i & 1) * W::kStage;
    const char* st = stage + own * W::kPair;
    const auto* m = reinterpret_cast<const typename L::M*>(stage + W::kMarks - W::kMarkFrom);
    const float4* hand = reinterpret_cast<const float4*>(smem + W::kHands + ((i & 1) * TILES + own) * W::kHand) + lane;
    sync();
    float w[MT][2][4];
    {
      // dW^T = (P^T do)^T + D^T (e^{B-b} K)^T
      float acc[MT][2][4] = {};
      uint32_t x[2][2][1][L::kHalves][4], s[2][2][MT][2][4];
      auto fetch = [&](int pair) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ks = 2 * pair + h;
#pragma unroll
          for (int k = 0; k < L::kHalves; ++k) load_block(x[pair & 1][h][0][k], st, ks * L::kHalves + k, lane);
#pragma unroll
          for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) a_rows<DK>(s[pair & 1][h][n][k], base + W::kState + k * W::kStatePlane, 16 * n, 16 * ks, lane);
        }
      };
      const float* scales = reinterpret_cast<const float*>(smem + W::kStateScale) + g * SIDES;
      fetch(0);
#pragma unroll
      for (int pair = 0; pair < SIDES / 2; ++pair) {
        if (pair + 1 < SIDES / 2) fetch(pair + 1);
        add_scaled<MT, 2, 2, L::kHalves>(acc, s[pair & 1], x[pair & 1], [&](int k, int n) {
          return make_float2(scales[16 * n * SIDES + 2 * pair + k], scales[(16 * n + 8) * SIDES + 2 * pair + k]);
        });
      }
      const float of_key = m->key;
      const float2 after[2] = {*reinterpret_cast<const float2*>(m->after + 16 * own + t), *reinterpret_cast<const float2*>(m->after + 16 * own + 8 + t)};
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 y = hand[32 * (n * (2 + 2 * SHARE) + j)];
          const float f0 = after[j].x * of_key, f1 = after[j].y * of_key;
          w[n][j][0] = fmaf(f0, acc[n][j][0], y.x); w[n][j][1] = fmaf(f1, acc[n][j][1], y.y);
          w[n][j][2] = fmaf(f0, acc[n][j][2], y.z); w[n][j][3] = fmaf(f1, acc[n][j][3], y.w);
        }
    }
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        float most = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) most = fmaxf(most, fabsf(w[n][e >> 1][2 * f + (e & 1)]));
        const Scale by = scale_of(over_row(most));
        const int row = 16 * n + g + 8 * f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t h[2];
          halves<2>(w[n][j][2 * f] * by.to, w[n][j][2 * f + 1] * by.to, h);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint32_t*>(smem + W::kW + k * W::kTokenPlane + unit_at<C>(row, 2 * own + j) + 2 * t) = h[k];
        }
        if ((lane & 3) == 0) reinterpret_cast<float*>(smem + W::kTokenScale)[row * TILES + own] = by.from;
      }
    const float total = m->total;
    sync();   // the planes of dW are there, those of D are read
#pragma unroll
    for (int n = 0; n < MT; ++n)
      if (16 * (tile0 + n) < p.d) {
        float4* to = reinterpret_cast<float4*>(p.im.dw + (chunk_of(i) * SIDES + tile0 + n) * L::kTokens + 2 * own * kBlock) + lane;
#pragma unroll
        for (int j = 0; j < 2; ++j) to[32 * j] = make_float4(w[n][j][0], w[n][j][1], w[n][j][2], w[n][j][3]);
      }
    if (!shares) continue;
    // D^T <- e^B D^T + (Q^T do)^T - dW^T K^, the chunk's part formed apart
    float sum[MT][2 * SHARE][4] = {};
    {
      uint32_t x[2][2][SHARE][2][4], v[2][2][MT][2][4];
      auto fetch = [&](int pair) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ks = 2 * pair + h;
#pragma unroll
          for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) a_rows<C>(v[pair & 1][h][n][k], base + W::kW + k * W::kTokenPlane, 16 * n, 16 * ks, lane);
#pragma unroll
          for (int j = 0; j < SHARE; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) load_block(x[pair & 1][h][j][k], st + W::kKeys, (j * TILES + ks) * 2 + k, lane);
        }
      };
      const float* scales = reinterpret_cast<const float*>(smem + W::kTokenScale) + g * TILES;
      fetch(0);
#pragma unroll
      for (int pair = 0; pair < TILES / 2; ++pair) {
        if (pair + 1 < TILES / 2) fetch(pair + 1);
        add_scaled<MT, 2 * SHARE, 2, 2>(sum, v[pair & 1], x[pair & 1], [&](int k, int n) {
          const float of_keys = m->keys[2 * pair + k];
          return make_float2(of_keys * scales[16 * n * TILES + 2 * pair + k], of_keys * scales[(16 * n + 8) * TILES + 2 * pair + k]);
        });
      }
    }
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j) {
        if (16 * (tile0 + n) < p.d)
          *reinterpret_cast<float4*>(p.im.ds + (chunk_of(i) * SIDES + tile0 + n) * L::kState + (2 * own * SHARE + j) * kBlock + 16 * lane) =
              make_float4(D[n][j][0], D[n][j][1], D[n][j][2], D[n][j][3]);
        const float4 x = hand[32 * (n * (2 + 2 * SHARE) + 2 + j)];
        const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) D[n][j][e] = fmaf(total, D[n][j][e], xs[e] - sum[n][j][e]);
      }
    publish();
  }
  if (shares && a.first) {
    float* first = a.first + bh * p.d * p.d;
#pragma unroll
    for (int n = 0; n < MT; ++n)
#pragma unroll
      for (int j = 0; j < 2 * SHARE; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * own * SHARE + 8 * j + t + (e & 1), c = 16 * (tile0 + n) + g + 8 * (e >> 1);
          if (r < p.d && c < p.d) first[static_cast<int64_t>(r) * p.d + c] = D[n][j][e];
        }
  }
}

struct GradArgs {
  Common c;
  Operand dq, dk, dv, dg, dbeta;   // dq, dk: of every value head when they are shared, float32 then
  uint32_t pairs;                  // stores of two values: 1 dq, 2 dk
};

template <typename T, int DK>
struct GradLay {
  using L = Lay<T, DK>;
  static constexpr int C = L::C, kStrips = C / 16, kWarps = 2 * kStrips, kThreads = 32 * kWarps;
  static constexpr int kHeld = (L::kSides + kWarps - 1) / kWarps;      // tiles of 16 value columns a warp
  static constexpr int kSlice = DK < 64 ? DK : 64;                     // columns of the values of a state at once
  static constexpr int kTurnedPlane = DK * C * 2, kTurned = L::kHalves * kTurnedPlane;   // planes [column][token]
  static constexpr int kSlicePlane = kSlice * DK * 2, kGrid = C + 8, kPairs = C * kGrid * 4, kSum = C * DK * 4;
  static constexpr int kPitch = DK + 4 / static_cast<int>(sizeof(T)), kValues = C * kPitch * static_cast<int>(sizeof(T));   // V, then dv, [token][column]
  static constexpr int kK = 0, kQ = kK + L::kInputHalf, kDout = kQ + L::kInputHalf, kW = kDout + L::kInputHalf, kR = kW + kTurned;
  static constexpr int kA = kR + kTurned;                              // T before it is A
  static constexpr int kL = kA + L::kInverse, kTurn = kL + L::kInverse, kState = kTurn + L::kInverse;   // A at its rows' scales, L, A at one scale
  static constexpr int kBytes = kState + std::max(L::kHalves * kSlicePlane, std::max(kValues, std::max(kPairs, kSum)));
  static_assert(kThreads == 4 * C, "four threads a token");
};

// Two values of row r, column tile n of planes W columns wide.
template <int W, int NH>
__device__ __forceinline__ void put(char* smem, int where, int plane, int r, int n, float x, float y) {
  uint32_t h[NH];
  halves<NH>(x, y, h);
#pragma unroll
  for (int k = 0; k < NH; ++k) *reinterpret_cast<uint32_t*>(smem + where + k * plane + unit_at<W>(r, n) + 4 * (threadIdx.x & 3)) = h[k];
}

// One chunk of one (b, h).  A pair of warps has 16 rows: one the products with dout (dq, A), the other those with dR (L, dk).
// Everything enters the tensor cores as one fp16 beside bf16 outputs (2^-11), two beside float32 ones, a whole plane at one scale.
template <typename T, int DK, typename O>
__global__ void __launch_bounds__(GradLay<T, DK>::kThreads, DK < 128 ? 2 : 1) delta_grads(const __grid_constant__ GradArgs a) {
  using G = GradLay<T, DK>;
  using L = Lay<T, DK>;
  constexpr int C = L::C, THREADS = G::kThreads, STRIPS = G::kStrips, NS = DK / 8, TILES = L::kSides, NH = L::kHalves, HELD = G::kHeld;
  extern __shared__ __align__(128) char smem[];
  __shared__ __align__(16) typename L::M m;
  __shared__ float vdot[TILES][C], rows_g[C], zk[C], parts[4][C], enters[2][C], leaves[C], crossing[C], both[G::kWarps];
  enum { kMostW, kMostR, kMostA, kMostL, kMostS, kMostD, kMosts };
  __shared__ uint32_t most[kMosts];   // the largest of each plane
  const Common& p = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t chunk = blockIdx.x % p.chunks;
  const int64_t bh = blockIdx.x / p.chunks, b = bh / p.H, h = bh % p.H;
  const int64_t at = bh * p.chunks + chunk, at_key = (b * p.Hk + h / (p.H / p.Hk)) * p.chunks + chunk;
  const int64_t t0 = static_cast<int64_t>(chunk) * C;
  const int rows = static_cast<int>(min(static_cast<int64_t>(C), p.N - t0));
  const uint32_t base = ptx::smem_u32(smem);
  const int g = lane >> 2, t = 2 * (lane & 3);
  const int strip = warp % STRIPS, m0 = 16 * strip, row = m0 + g;
  const bool second = warp >= STRIPS;

  copy_async(base + G::kK, p.im.k + at_key * L::kInputHalf, L::kInputHalf, threadIdx.x, THREADS);
  copy_async(base + G::kQ, p.im.q + at_key * L::kInputHalf, L::kInputHalf, threadIdx.x, THREADS);
  copy_async(base + G::kDout, p.im.dout + at * L::kInputHalf, L::kInputHalf, threadIdx.x, THREADS);
  copy_async(base + G::kA, p.im.inverse + at * L::kInverse, L::kInverse, threadIdx.x, THREADS);
  copy_async(ptx::smem_u32(&m), p.im.marks + at * L::kMarks, L::kMarks, threadIdx.x, THREADS);
  commit();
  T* values = reinterpret_cast<T*>(smem + G::kState);
  {
    const T* v = static_cast<const T*>(p.v.data) + b * p.v.sb + h * p.v.sh + t0 * p.v.sn;
    const T zero = T(0.0f);
#pragma unroll 8
    for (int i = threadIdx.x; i < C * DK; i += THREADS) {
      const int r = i / DK, c = i % DK;
      values[r * G::kPitch + c] = r < rows && c < p.d ? v[r * p.v.sn + c] : zero;
    }
  }
  if (threadIdx.x < kMosts) most[threadIdx.x] = 0;
  __syncthreads();
  auto note = [&](int which, float largest) {
    const uint32_t all = __reduce_max_sync(~0u, __float_as_uint(largest));
    if (lane == 0) atomicMax(most + which, all);
  };
  auto scale = [&](int which) { return plane_scale(most[which]); };
  auto size = [](float4 x) { return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))); };
  // fragments of W and dW; <S, D> and the largest of both states
  float4 w[HELD][C / 8], dw[HELD][C / 8];
  const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float through = 0.0f;
  {
    float of_w = 0.0f, of_s = 0.0f, of_d = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int tile = warp + i * G::kWarps;
      const bool in = 16 * tile < p.d;
      const float4 *from = reinterpret_cast<const float4*>(p.im.w + (at * TILES + tile) * L::kTokens) + lane,
                   *from_d = reinterpret_cast<const float4*>(p.im.dw + (at * TILES + tile) * L::kTokens) + lane;
#pragma unroll
      for (int n = 0; n < C / 8; ++n) {
        w[i][n] = in ? from[32 * n] : none;
        dw[i][n] = in ? from_d[32 * n] : none;
      }
    }
    const int64_t off = at * TILES * L::kState;
    const int used = (p.d + 15) / 16 * NS * 32;   // float4 of either state
#pragma unroll 4
    for (int i = threadIdx.x; i < used; i += THREADS) {
      const float4 x = reinterpret_cast<const float4*>(p.im.s + off)[i], y = reinterpret_cast<const float4*>(p.im.ds + off)[i];
      of_s = fmaxf(of_s, size(x));
      of_d = fmaxf(of_d, size(y));
      through = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, through))));
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i)
#pragma unroll
      for (int n = 0; n < C / 8; ++n) of_w = fmaxf(of_w, size(w[i][n]));
    note(kMostW, of_w);
    note(kMostS, of_s);
    note(kMostD, of_d);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) through += __shfl_xor_sync(~0u, through, o);
    if (lane == 0) both[warp] = through;
  }
  wait_all();
  __syncthreads();

  // W's planes; dR^T = dW^T T, each row of dW^T at its own scale; dv; dR . V
  {
    const Scale by_w = scale(kMostW);
    float of_r = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int tile = warp + i * G::kWarps;
      if (tile >= TILES) break;
      float largest[2] = {0.0f, 0.0f};
#pragma unroll
      for (int n = 0; n < C / 8; ++n) {
        const float4 x = w[i][n], y = dw[i][n];
        put<C, NH>(smem, G::kW, G::kTurnedPlane, 16 * tile + g, n, x.x * by_w.to, x.y * by_w.to);
        put<C, NH>(smem, G::kW, G::kTurnedPlane, 16 * tile + g + 8, n, x.z * by_w.to, x.w * by_w.to);
        largest[0] = fmaxf(largest[0], fmaxf(fabsf(y.x), fabsf(y.y)));
        largest[1] = fmaxf(largest[1], fmaxf(fabsf(y.z), fabsf(y.w)));
      }
      const Scale by[2] = {scale_of(over_row(largest[0])), scale_of(over_row(largest[1]))};
      float acc[C / 8][4] = {};
#pragma unroll
      for (int ks = 0; ks < STRIPS; ++ks) {
        uint32_t x[NH][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float4 y = dw[i][2 * ks + n];
          uint32_t h2[NH];
          halves<NH>(y.x * by[0].to, y.y * by[0].to, h2);
#pragma unroll
          for (int k = 0; k < NH; ++k) x[k][2 * n] = h2[k];
          halves<NH>(y.z * by[1].to, y.w * by[1].to, h2);
#pragma unroll
          for (int k = 0; k < NH; ++k) x[k][2 * n + 1] = h2[k];
        }
#pragma unroll
        for (int s = 0; s <= ks; ++s) {
          uint32_t y[NH][4];
#pragma unroll
          for (int k = 0; k < NH; ++k) b_cols<C>(y[k], base + G::kA + k * L::kSquare, 16 * s, 16 * ks, lane);
#pragma unroll
          for (int f = 0; f < 2; ++f) add_products(acc[2 * s + f], x, y, f);
        }
      }
      const float f0 = by[0].from * m.inverse, f1 = by[1].from * m.inverse;
#pragma unroll
      for (int n = 0; n < C / 8; ++n) {
        const float4 x = make_float4(acc[n][0] * f0, acc[n][1] * f0, acc[n][2] * f1, acc[n][3] * f1);
        dw[i][n] = x;
        of_r = fmaxf(of_r, size(x));
        const float xs[4] = {x.x, x.y, x.z, x.w};
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int token = 8 * n + t + (e & 1);
          T* v = values + token * G::kPitch + 16 * tile + g + 8 * (e >> 1);
          sum[e & 1] = fmaf(xs[e], to_f(*v), sum[e & 1]);
          from_f(v, m.beta[token] * xs[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sum[e] += __shfl_xor_sync(~0u, sum[e], 4);
          sum[e] += __shfl_xor_sync(~0u, sum[e], 8);
          sum[e] += __shfl_xor_sync(~0u, sum[e], 16);
          if (lane < 4) vdot[tile][8 * n + t + e] = sum[e];
        }
      }
    }
    note(kMostR, of_r);
  }
  __syncthreads();
  {
    T* dv = static_cast<T*>(a.dv.data) + b * a.dv.sb + h * a.dv.sh + t0 * a.dv.sn;
    for (int i = threadIdx.x; i < C * DK; i += THREADS) {
      const int r = i / DK, c = i % DK;
      if (r < rows && c < p.d) dv[r * a.dv.sn + c] = values[r * G::kPitch + c];
    }
    const float by = scale(kMostR).to;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int tile = warp + i * G::kWarps;
      if (tile >= TILES) break;
#pragma unroll
      for (int n = 0; n < C / 8; ++n) {
        const float4 x = dw[i][n];
        put<C, NH>(smem, G::kR, G::kTurnedPlane, 16 * tile + g, n, x.x * by, x.y * by);
        put<C, NH>(smem, G::kR, G::kTurnedPlane, 16 * tile + g + 8, n, x.z * by, x.w * by);
      }
    }
  }
  __syncthreads();

  // do W^T and Q K^T (first), dR W^T and K K^T (second), up to the diagonal: A and L, and the pairs of the gates
  const float of_w = scale(kMostW).from, of_r = scale(kMostR).from;
  float kept[2 * STRIPS][4], pairs[2 * STRIPS][4];
  Scale of_row[2] = {};
  {
    float x[2 * STRIPS][4] = {}, y[2 * STRIPS][4] = {};
#pragma unroll 1
    for (int ks = 0; ks < TILES; ++ks) {
      uint32_t l[NH][4], key[NH][4];
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        a_rows<DK>(key[n], base + (second ? G::kK : G::kQ) + n * L::kRows, m0, 16 * ks, lane);
        if (second)
          a_cols<C>(l[n], base + G::kR + n * G::kTurnedPlane, m0, 16 * ks, lane);
        else
          a_rows<DK>(l[n], base + G::kDout + n * L::kRows, m0, 16 * ks, lane);
      }
#pragma unroll
      for (int s = 0; s < STRIPS; ++s) {
        if (s > strip) continue;
        uint32_t u[NH][4], k[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
          b_cols<C>(u[n], base + G::kW + n * G::kTurnedPlane, 16 * s, 16 * ks, lane);
          b_rows<DK>(k[n], base + G::kK + n * L::kRows, 16 * s, 16 * ks, lane);
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          add_products(x[2 * s + f], l, u, f);
          add_products(y[2 * s + f], key, k, f);
        }
      }
    }
    const float of_x[2] = {of_w * (second ? of_r : m.douts[row]), of_w * (second ? of_r : m.douts[row + 8])}, of_y = m.key * (second ? m.key : m.queries);
    const Sum br[2] = {{m.hi[row], m.lo[row]}, {m.hi[row + 8], m.lo[row + 8]}};
    const float beta_r[2] = {m.beta[row], m.beta[row + 8]};
    float sum[2] = {0.0f, 0.0f}, largest[2] = {0.0f, 0.0f};
#pragma unroll
    for (int n = 0; n < 2 * STRIPS; ++n) {
      const int c = 8 * n + t;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = row + 8 * (e >> 1), s = c + (e & 1);
        kept[n][e] = pairs[n][e] = 0.0f;
        if (n >= 2 * strip + 2) continue;
        const Sum bc = {m.hi[s], m.lo[s]};
        const float decay = s <= r ? exp2_of(br[e >> 1], bc) : 0.0f;
        const float d = s <= r ? x[n][e] * of_x[e >> 1] * decay : 0.0f, k = y[n][e] * of_y;
        if (second) {
          kept[n][e] = s < r ? -beta_r[e >> 1] * d : 0.0f;
          if (s < r) sum[e >> 1] = fmaf(d, k, sum[e >> 1]);
        } else {
          kept[n][e] = p.scale * d;
        }
        pairs[n][e] = s < r ? kept[n][e] * k : 0.0f;
        largest[e >> 1] = fmaxf(largest[e >> 1], fabsf(kept[n][e]));
      }
    }
    note(second ? kMostL : kMostA, fmaxf(largest[0], largest[1]));
#pragma unroll
    for (int f = 0; f < 2; ++f) of_row[f] = plane_scale(__float_as_uint(over_row(largest[f])));
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      sum[f] += __shfl_xor_sync(~0u, sum[f], 1);
      sum[f] += __shfl_xor_sync(~0u, sum[f], 2);
      if (second && (lane & 3) == 0) rows_g[row + 8 * f] = sum[f];
    }
  }
  // pairs that a gate lies between: sums over the rows from the gate on, then over the columns in front of it
  float* grid = reinterpret_cast<float*>(smem + G::kState);
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    if (second == (turn == 1))
#pragma unroll
      for (int n = 0; n < 2 * STRIPS; ++n)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float2* to = reinterpret_cast<float2*>(grid + (row + 8 * f) * G::kGrid + 8 * n + t);
          float2 x = make_float2(pairs[n][2 * f], pairs[n][2 * f + 1]);
          if (turn) x = make_float2(to->x + x.x, to->y + x.y);
          *to = x;
        }
    if (turn == 1) {   // every warp's largest is noted; T's planes, where A goes, were last read long ago
      const float by = scale(second ? kMostL : kMostA).to;
#pragma unroll
      for (int n = 0; n < 2 * STRIPS; ++n) {
        if (n >= 2 * strip + 2) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          put<C, NH>(smem, second ? G::kL : G::kTurn, L::kSquare, row + 8 * e, n, kept[n][2 * e] * by, kept[n][2 * e + 1] * by);
          if (!second) put<C, NH>(smem, G::kA, L::kSquare, row + 8 * e, n, kept[n][2 * e] * of_row[e].to, kept[n][2 * e + 1] * of_row[e].to);
        }
      }
    }
    __syncthreads();
  }
  {
    constexpr int PART = C / 4;   // a thread's rows of a column, then columns of a row
    const int c = threadIdx.x % C, r0 = threadIdx.x / C * PART;
    float run[PART];
#pragma unroll
    for (int i = 0; i < PART; ++i) run[i] = grid[(r0 + i) * G::kGrid + c];
#pragma unroll
    for (int i = PART - 2; i >= 0; --i) run[i] += run[i + 1];
    parts[threadIdx.x / C][c] = run[0];
    __syncthreads();
    float behind = 0.0f;
#pragma unroll
    for (int j = 3; j > 0; --j)
      if (j * PART > r0) behind += parts[j][c];
#pragma unroll
    for (int i = 0; i < PART; ++i) grid[(r0 + i) * G::kGrid + c] = run[i] + behind;
    __syncthreads();
    const int r = threadIdx.x / 4, c0 = (threadIdx.x & 3) * PART;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PART; ++i) {   // each row from another column on: the lanes at other banks
      const int s = c0 + ((i + r) & (PART - 1));
      sum += s < r ? grid[r * G::kGrid + s] : 0.0f;
    }
    sum += __shfl_xor_sync(~0u, sum, 1);
    sum += __shfl_xor_sync(~0u, sum, 2);
    if ((threadIdx.x & 3) == 0) crossing[r] = sum;
  }
  __syncthreads();

  const float of_a = scale(kMostA).from, of_l = scale(kMostL).from;
  float acc[NS][4] = {};
  // rows of S^T or D^T of a slice of the values' columns
  auto fill = [&](const char* from, int slice, float by) {
    for (int j = warp; j < G::kSlice / 16 * NS; j += G::kWarps) {
      const int tile = slice * (G::kSlice / 16) + j / NS, n = j % NS;
      const float4 x = 16 * tile < p.d ? reinterpret_cast<const float4*>(from + (at * TILES + tile) * L::kState)[32 * n + lane] : none;
      const int r = 16 * (j / NS) + g;
      put<DK, NH>(smem, G::kState, G::kSlicePlane, r, n, x.x * by, x.y * by);
      put<DK, NH>(smem, G::kState, G::kSlicePlane, r + 8, n, x.z * by, x.w * by);
    }
  };
  // a row's sum of acc times the rows of a plane
  auto dot_rows = [&](int where, float of_plane, float (&sum)[2]) {
    sum[0] = sum[1] = 0.0f;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        float2 x = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = NH - 1; k >= 0; --k) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(smem + where + k * L::kRows + unit_at<DK>(row + 8 * f, n) + 2 * t));
          x.x += y.x;
          x.y += y.y;
        }
        sum[f] = fmaf(acc[n][2 * f], x.x, fmaf(acc[n][2 * f + 1], x.y, sum[f]));
      }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      sum[f] += __shfl_xor_sync(~0u, sum[f], 1);
      sum[f] += __shfl_xor_sync(~0u, sum[f], 2);
      sum[f] *= of_plane;
    }
  };
  // acc += (f0, f1 of the rows) times 16 rows of KS steps of k, those from `from` up to `to`, with planes [k][channel]
  auto add_rows = [&](const auto& l, int from, int to, int where, int plane, float f0, float f1) {
    constexpr int STEPS = sizeof(l) / (NH * 16);
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) {
      float c[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < STEPS; ++ks) {
        if (ks < from || ks >= to) continue;
        uint32_t x[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n) b_cols<DK>(x[n], base + where + n * plane, 16 * j, 16 * ks, lane);
#pragma unroll
        for (int f = 0; f < 2; ++f) add_products(c[f], l[ks], x, f);
      }
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[2 * j + f][e] = fmaf(c[f][e], e < 2 ? f0 : f1, acc[2 * j + f][e]);
    }
  };
  // rows of a square plane, or of its transpose, times the rows of an input
  auto add_square = [&](int square, bool turned, int where, float f0, float f1) {
    uint32_t l[STRIPS][NH][4];
#pragma unroll
    for (int ks = 0; ks < STRIPS; ++ks) {
      if (turned ? ks < strip : ks > strip) continue;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (turned)
          a_cols<C>(l[ks][n], base + square + n * L::kSquare, m0, 16 * ks, lane);
        else
          a_rows<C>(l[ks][n], base + square + n * L::kSquare, m0, 16 * ks, lane);
      }
    }
    add_rows(l, turned ? strip : 0, turned ? STRIPS : strip + 1, where, L::kRows, f0, f1);
  };
  // rows of dout, or of the transposes of dR, W, times the state's slice
  auto add_state = [&](int slice, int turned, float f0, float f1) {
    constexpr int STEPS = G::kSlice / 16;
    uint32_t l[STEPS][NH][4];
#pragma unroll
    for (int ks = 0; ks < STEPS; ++ks) {
      const int k0 = slice * G::kSlice + 16 * ks;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (turned)
          a_cols<C>(l[ks][n], base + turned + n * G::kTurnedPlane, m0, k0, lane);
        else
          a_rows<DK>(l[ks][n], base + G::kDout + n * L::kRows, m0, k0, lane);
      }
    }
    add_rows(l, 0, STEPS, G::kState, G::kSlicePlane, f0, f1);
  };
  auto store = [&](const Operand& to, bool two) {
    O* out = static_cast<O*>(to.data) + b * to.sb + h * to.sh + t0 * to.sn;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int r = row + 8 * f;
      if (r >= rows) continue;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        const int c = 8 * n + t;
        if (c < p.d) store_pair<O>(out + r * to.sn + c, acc[n][2 * f], acc[n][2 * f + 1], two, c + 1 < p.d);
      }
    }
  };

  const float in0 = m.inside[row], in1 = m.inside[row + 8];
  const Scale by_s = scale(kMostS), by_d = scale(kMostD);
  for (int slice = 0; slice < DK / G::kSlice; ++slice) {
    fill(p.im.s, slice, by_s.to);
    __syncthreads();
    if (second)
      add_state(slice, G::kR, of_r * by_s.from, of_r * by_s.from);
    else
      add_state(slice, 0, p.scale * in0 * m.douts[row] * by_s.from, p.scale * in1 * m.douts[row + 8] * by_s.from);
    __syncthreads();
  }
  {
    float sum[2];
    if (second) {
      dot_rows(G::kK, m.key, sum);
      const float b0 = -m.beta[row] * in0, b1 = -m.beta[row + 8] * in1;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] *= e < 2 ? b0 : b1;
      if ((lane & 3) == 0) {
        zk[row] = in0 * sum[0];
        zk[row + 8] = in1 * sum[1];
        enters[1][row] = b0 * sum[0];
        enters[1][row + 8] = b1 * sum[1];
      }
      add_square(G::kL, false, G::kK, of_l * m.key, of_l * m.key);
      add_square(G::kL, true, G::kK, of_l * m.key, of_l * m.key);
    } else {
      dot_rows(G::kQ, m.queries, sum);
      if ((lane & 3) == 0) {
        enters[0][row] = sum[0];
        enters[0][row + 8] = sum[1];
      }
      add_square(G::kA, false, G::kK, of_row[0].from * m.key, of_row[1].from * m.key);
      store(a.dq, a.pairs & 1);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
    }
  }
  for (int slice = 0; slice < DK / G::kSlice; ++slice) {
    fill(p.im.ds, slice, by_d.to);
    __syncthreads();
    if (!second) add_state(slice, G::kW, m.after[row] * of_w * by_d.from, m.after[row + 8] * of_w * by_d.from);
    __syncthreads();
  }
  float4* half = reinterpret_cast<float4*>(smem + G::kState) + strip * NS * 32 + lane;
  if (!second) {
    float sum[2];
    dot_rows(G::kK, m.key, sum);
    if ((lane & 3) == 0) {
      leaves[row] = sum[0];
      leaves[row + 8] = sum[1];
    }
    add_square(G::kTurn, true, G::kQ, of_a * m.queries, of_a * m.queries);
#pragma unroll
    for (int n = 0; n < NS; ++n) half[32 * n] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  }
  __syncthreads();
  if (second) {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const float4 x = half[32 * n];
      acc[n][0] += x.x; acc[n][1] += x.y; acc[n][2] += x.z; acc[n][3] += x.w;
    }
    store(a.dk, a.pairs & 2);
  }
  constexpr int PART = C / 4;
  const int token = threadIdx.x / 4, s0 = (threadIdx.x & 3) * PART;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < PART; ++i) sum += s0 + i >= token ? enters[0][s0 + i] + enters[1][s0 + i] : leaves[s0 + i];
  sum += __shfl_xor_sync(~0u, sum, 1);
  sum += __shfl_xor_sync(~0u, sum, 2);
  if ((threadIdx.x & 3) == 0 && token < rows) {
    float dbeta = 0.0f, all = 0.0f;
#pragma unroll
    for (int n = 0; n < TILES; ++n) dbeta += vdot[n][token];
    dbeta -= zk[token] + rows_g[token];
#pragma unroll
    for (int n = 0; n < G::kWarps; ++n) all += both[n];
    const float dg = fmaf(m.total, all, crossing[token] + sum);
    from_f(static_cast<T*>(a.dg.data) + b * a.dg.sb + h * a.dg.sh + (t0 + token) * a.dg.sn, dg);
    from_f(static_cast<T*>(a.dbeta.data) + b * a.dbeta.sb + h * a.dbeta.sh + (t0 + token) * a.dbeta.sn, dbeta);
  }
}

// Gradients of shared heads: the sum over the value heads of each, in their order.
struct Shared {
  const float* part[2];   // [B][N][H][d]
  Operand to[2];
  int64_t N, total;       // elements of one of them
  int32_t Hk, times, d;
};
template <typename T>
__global__ void __launch_bounds__(256) delta_shared(const __grid_constant__ Shared a) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.total) return;
  const int c = static_cast<int>(i % a.d);
  const int64_t head = i / a.d, hk = head % a.Hk, token = head / a.Hk, n = token % a.N, b = token / a.N;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const float* x = a.part[o] + head * a.times * a.d + c;
    float sum = 0.0f;
    for (int j = 0; j < a.times; ++j) sum += x[static_cast<int64_t>(j) * a.d];
    from_f(static_cast<T*>(a.to[o].data) + b * a.to[o].sb + n * a.to[o].sn + hk * a.to[o].sh + c, sum);
  }
}

template <typename T, int DK, int MT>
int back_as(const BackArgs& a, int64_t BH, cudaStream_t s) {
  using W = BackLay<T, DK, MT>;
  static_assert(W::kBytes <= 227 * 1024, "shared memory");
  if (cudaFuncSetAttribute(delta_back<T, DK, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  const int groups = (a.c.d + 16 * MT - 1) / (16 * MT);
  KernelTimer timer("delta_back", s);
  delta_back<T, DK, MT><<<static_cast<unsigned>(BH * groups), W::kThreads, W::kBytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK, typename O>
int grads_as(const GradArgs& a, int64_t BH, cudaStream_t s) {
  using G = GradLay<T, DK>;
  static_assert(G::kBytes <= 220 * 1024, "shared memory");
  if (cudaFuncSetAttribute(delta_grads<T, DK, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kBytes) != cudaSuccess)
    return MHLA_ERR_CUDA;
  KernelTimer timer("delta_grads", s);
  delta_grads<T, DK, O><<<static_cast<unsigned>(BH * a.c.chunks), G::kThreads, G::kBytes, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

template <typename T, int DK>
int run_as(const BackArgs& b, const GradArgs& g, int64_t BH, bool shared, cudaStream_t s) {
  int rc;
  if constexpr (DK == 64)
    rc = two_tiles(BH, b.c.d, sizeof(T) == 2 ? kSms : 2 * kSms) ? back_as<T, DK, 2>(b, BH, s) : back_as<T, DK, 1>(b, BH, s);
  else
    rc = back_as<T, DK, 1>(b, BH, s);
  if (rc != MHLA_OK) return rc;
  return shared && sizeof(T) == 2 ? grads_as<T, DK, float>(g, BH, s) : grads_as<T, DK, T>(g, BH, s);
}

template <typename T>
int run_type(const BackArgs& b, const GradArgs& g, int64_t BH, bool shared, cudaStream_t s) {
  switch (padded(b.c.d)) {
    case 32: return run_as<T, 32>(b, g, BH, shared, s);
    case 64: return run_as<T, 64>(b, g, BH, shared, s);
    default: return run_as<T, 128>(b, g, BH, shared, s);
  }
}

size_t shared_bytes(const DeltaProblem& p) { return p.H == p.Hk ? 0 : align_up(static_cast<size_t>(p.B * p.N * p.H * p.d) * 4); }

}  // namespace

size_t delta_bwd_workspace_bytes(const DeltaProblem& p) {
  Images im;
  return lay_out(p, true, nullptr, &im) + 2 * shared_bytes(p);
}

int launch_delta_backward(const DeltaProblem& p, const DeltaBackward& d, void* workspace, void* stream) {
  ScanArgs a = {};
  a.c = common(p, &d.dout);
  char* rest = static_cast<char*>(workspace);
  rest += lay_out(p, true, rest, &a.c.im);
  a.init = d.state_in;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t BH = p.B * p.H;
  int rc = launch_prepare(a.c, BH, p.dtype, true, s);
  if (rc == MHLA_OK) rc = launch_scan(a, BH, p.dtype, true, s);
  if (rc != MHLA_OK) return rc;
  const BackArgs b = {a.c, d.dstate_out, d.dstate_in};
  GradArgs g = {a.c, d.dq, d.dk, d.dv, d.dg, d.dbeta, 0};
  const bool shared = p.H != p.Hk;
  float* part[2] = {reinterpret_cast<float*>(rest), reinterpret_cast<float*>(rest + shared_bytes(p))};
  if (shared) {
    g.dq = Operand{part[0], p.N * p.H * p.d, p.H * p.d, p.d};
    g.dk = Operand{part[1], p.N * p.H * p.d, p.H * p.d, p.d};
  }
  const int dtype = shared ? MHLA_F32 : p.dtype;
  g.pairs = (pairs_fit(g.dq, p.d, dtype) ? 1u : 0u) | (pairs_fit(g.dk, p.d, dtype) ? 2u : 0u);
  rc = p.dtype == MHLA_BF16 ? run_type<__nv_bfloat16>(b, g, BH, shared, s) : run_type<float>(b, g, BH, shared, s);
  if (rc != MHLA_OK || !shared) return rc;
  Shared sh = {{part[0], part[1]}, {d.dq, d.dk}, p.N, p.B * p.N * p.Hk * p.d, static_cast<int32_t>(p.Hk),
               static_cast<int32_t>(p.H / p.Hk), p.d};
  KernelTimer timer("delta_shared", s);
  const unsigned grid = static_cast<unsigned>((sh.total + 255) / 256);
  if (p.dtype == MHLA_BF16)
    delta_shared<__nv_bfloat16><<<grid, 256, 0, s>>>(sh);
  else
    delta_shared<float><<<grid, 256, 0, s>>>(sh);
  return cudaGetLastError() == cudaSuccess ? MHLA_OK : MHLA_ERR_CUDA;
}

int read_and_clear_delta_back_error(void* stream, uint32_t* flags) {
  return tc::read_and_clear_word(g_delta_back_error, stream, flags);
}

MHLA_DEFINE_STALL_SETTER(set_stall_delta_back)

}  // namespace mhla
