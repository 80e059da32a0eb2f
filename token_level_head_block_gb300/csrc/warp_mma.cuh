// Products of small tiles on mma.sync (bf16 terms, float32 accumulators), what feeds them from shared
// memory, and the layout of tiles there.
#pragma once

#include <cstdint>

namespace mhla {
namespace gated {

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

// The same products of fp16 operands.
__device__ __forceinline__ void mma_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_half_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// Byte offset of a 16-byte unit of a row-major bf16 tile W columns wide.  Units change
// places with the row's number, so that eight rows read at one column (ldmatrix) or
// written at one (accumulators) meet all banks.
template <int W>
__device__ __forceinline__ int unit_at(int row, int unit) {
  return row * (2 * W) + ((unit ^ (W == 32 ? (row >> 1) & 3 : row & 7)) << 4);
}

// Operands of 16 rows (A) or 16 columns (B, two column tiles) by 16 of k, from planes W columns wide.
template <int W>
__device__ __forceinline__ void a_rows(uint32_t (&a)[4], uint32_t base, int m0, int k0, int lane) {   // [m][k]
  ldsm(a, base + unit_at<W>(m0 + (lane & 7) + ((lane >> 3) & 1) * 8, (k0 >> 3) + (lane >> 4)));
}
template <int W>
__device__ __forceinline__ void a_cols(uint32_t (&a)[4], uint32_t base, int m0, int k0, int lane) {   // [k][m]
  ldsm_t(a, base + unit_at<W>(k0 + (lane & 7) + (lane >> 4) * 8, (m0 >> 3) + ((lane >> 3) & 1)));
}
template <int W>
__device__ __forceinline__ void b_rows(uint32_t (&b)[4], uint32_t base, int n0, int k0, int lane) {   // [n][k]
  ldsm(b, base + unit_at<W>(n0 + (lane & 7) + (lane >> 4) * 8, (k0 >> 3) + ((lane >> 3) & 1)));
}
template <int W>
__device__ __forceinline__ void b_cols(uint32_t (&b)[4], uint32_t base, int n0, int k0, int lane) {   // [k][n]
  ldsm_t(b, base + unit_at<W>(k0 + (lane & 7) + ((lane >> 3) & 1) * 8, (n0 >> 3) + (lane >> 4)));
}

}  // namespace gated
}  // namespace mhla
