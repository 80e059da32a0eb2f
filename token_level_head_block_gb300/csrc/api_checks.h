// Host-side argument checks the entry points share: dtypes, spans of strided
// [B, N, H, d] tensors and their overlaps.
#pragma once

#include <algorithm>
#include <cstdint>
#include <utility>

#include "../../include/mhla.h"

namespace mhla {

inline int64_t elem_bytes(int dtype) { return dtype == MHLA_BF16 ? 2 : 4; }

inline bool valid_dtype(int dtype) { return dtype == MHLA_BF16 || dtype == MHLA_F32; }

// Byte span [lo, hi) a [B, N, H, d] tensor can touch.
inline void span(const mhla_tensor_t* t, uintptr_t* lo, uintptr_t* hi) {
  const int64_t e = elem_bytes(t->dtype);
  const int64_t last = (t->B - 1) * t->stride_b + (t->N - 1) * t->stride_n + (t->H - 1) * t->stride_h + t->d;
  *lo = reinterpret_cast<uintptr_t>(t->data);
  *hi = *lo + static_cast<uintptr_t>(last * e);
}

inline bool overlaps(uintptr_t a0, uintptr_t a1, uintptr_t b0, uintptr_t b1) { return a0 < b1 && b0 < a1; }

// No two (b, n, h, c) index tuples of an output may share an address: sort the
// three outer dimensions by stride and require each stride to clear the extent
// of everything inside it.
inline bool non_overlapping(const mhla_tensor_t* t) {
  struct Dim { int64_t stride, extent; } dims[3] = {
      {t->stride_b, t->B}, {t->stride_n, t->N}, {t->stride_h, t->H}};
  std::sort(dims, dims + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  int64_t inner = t->d;   // elements spanned so far
  for (const Dim& dm : dims) {
    if (dm.extent <= 1) continue;
    if (dm.stride < inner) return false;
    inner = dm.stride * (dm.extent - 1) + inner;
  }
  return true;
}

inline int check_tensor(const mhla_tensor_t* t) {
  if (!t) return MHLA_ERR_INVALID_ARG;
  if (!valid_dtype(t->dtype)) return MHLA_ERR_INVALID_ARG;
  if (t->B < 0 || t->N < 1 || t->H < 0 || t->d < 1 || t->d > 128) return MHLA_ERR_INVALID_ARG;
  if (t->stride_b < 0 || t->stride_n < 0 || t->stride_h < 0) return MHLA_ERR_INVALID_ARG;
  if (t->B > 0 && t->H > 0 && !t->data) return MHLA_ERR_INVALID_ARG;
  return MHLA_OK;
}

inline bool same_shape(const mhla_tensor_t* a, const mhla_tensor_t* b) {
  return a->B == b->B && a->N == b->N && a->H == b->H && a->d == b->d && a->dtype == b->dtype;
}

struct Axis {
  int64_t stride, extent;
};

// Two runs of elements, [0, la) and [off, off + lb), repeated along the same
// axes, never meet: off >= la, and every stride clears what lies inside it.
inline bool runs_apart(int64_t off, int64_t la, int64_t lb, Axis* axes, int count) {
  if (off < la) return false;
  std::sort(axes, axes + count, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
  int64_t inner = off + lb;
  for (int i = 0; i < count; ++i) {
    if (axes[i].extent <= 1) continue;
    if (axes[i].stride < inner) return false;
    inner += axes[i].stride * (axes[i].extent - 1);
  }
  return true;
}

// Whether two non-empty tensors of the same B and N share no element: their
// spans are apart, or they are views of one buffer that lie side by side in
// every token's row (q and k in a projection's [B, N, 3C]) or in every head's.
inline bool disjoint(const mhla_tensor_t* a, const mhla_tensor_t* b) {
  uintptr_t a0, a1, b0, b1;
  span(a, &a0, &a1);
  span(b, &b0, &b1);
  if (!overlaps(a0, a1, b0, b1)) return true;
  if (a0 > b0) {
    std::swap(a, b);
    std::swap(a0, b0);
  }
  const int64_t e = elem_bytes(a->dtype);
  if (a->dtype != b->dtype || (b0 - a0) % e != 0) return false;
  if ((a->N > 1 && a->stride_n != b->stride_n) || (a->B > 1 && a->stride_b != b->stride_b)) return false;
  const int64_t off = static_cast<int64_t>(b0 - a0) / e;
  Axis rows[2] = {{a->stride_n, a->N}, {a->stride_b, a->B}};
  if (runs_apart(off, (a->H - 1) * a->stride_h + a->d, (b->H - 1) * b->stride_h + b->d, rows, 2)) return true;
  if (a->stride_h != b->stride_h) return false;
  Axis heads[3] = {{a->stride_n, a->N}, {a->stride_b, a->B}, {a->stride_h, std::max(a->H, b->H)}};
  return runs_apart(off, a->d, b->d, heads, 3);
}

inline bool same_view(const mhla_tensor_t* a, const mhla_tensor_t* b) {
  return a->data == b->data && a->dtype == b->dtype && a->B == b->B && a->N == b->N && a->H == b->H && a->d == b->d &&
         a->stride_b == b->stride_b && a->stride_n == b->stride_n && a->stride_h == b->stride_h;
}

// Whether the tensor's span meets `bytes` bytes of plain memory at p.
inline bool meets(const mhla_tensor_t* t, const void* p, int64_t bytes) {
  uintptr_t t0, t1;
  span(t, &t0, &t1);
  const uintptr_t p0 = reinterpret_cast<uintptr_t>(p);
  return p && overlaps(t0, t1, p0, p0 + static_cast<uintptr_t>(bytes));
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace mhla
