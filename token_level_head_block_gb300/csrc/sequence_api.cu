// extern "C" entry points of the gated recurrence, of the gated delta rule, of the query/key norm
// with rotation and of the linear layer around them: argument checks, workspace handling, launches.  Every check
// runs on the host before anything is queued on the stream.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "mhla_internal.h"

namespace mhla {
namespace {

bool empty(const mhla_tensor_t* t) { return t->B == 0 || t->H == 0; }

// What every tensor of these calls must be: a sound description at an address its elements may have.
int check_elements(const mhla_tensor_t* t) {
  const int rc = check_tensor(t);
  if (rc != MHLA_OK) return rc;
  return reinterpret_cast<uintptr_t>(t->data) % elem_bytes(t->dtype) == 0 ? MHLA_OK : MHLA_ERR_INVALID_ARG;
}

Operand operand(const mhla_tensor_t* t) { return Operand{t->data, t->stride_b, t->stride_n, t->stride_h}; }

// The [B, N, H, 1] companion of q.
bool gate_shape(const mhla_tensor_t* q, const mhla_tensor_t* g) {
  return g->B == q->B && g->N == q->N && g->H == q->H && g->d == 1 && g->dtype == q->dtype;
}

int64_t state_bytes(const mhla_tensor_t* q) { return q->B * q->H * q->d * q->d * int64_t{4}; }

bool plain_overlap(const void* a, const void* b, int64_t bytes, int64_t bytes_b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && overlaps(x, x + static_cast<uintptr_t>(bytes), y, y + static_cast<uintptr_t>(bytes_b));
}
bool plain_overlap(const void* a, const void* b, int64_t bytes) { return plain_overlap(a, b, bytes, bytes); }

// Each CTA owns (b, h) and a span of tokens; b, h and the span fit one 31-bit
// grid axis.
int check_gated(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v, const mhla_tensor_t* g,
                float scale) {
  for (const mhla_tensor_t* t : {q, k, v, g}) {
    const int rc = check_elements(t);
    if (rc != MHLA_OK) return rc;
  }
  if (!same_shape(q, k) || !same_shape(q, v) || !gate_shape(q, g)) return MHLA_ERR_SHAPE;
  if (!std::isfinite(scale)) return MHLA_ERR_INVALID_ARG;
  if (q->N > (int64_t{1} << 40) || q->B > (int64_t{1} << 24) || q->H > (int64_t{1} << 24) ||
      q->B * q->H > (int64_t{1} << 24))
    return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

// A written tensor: no element twice, none shared with the others given, none
// inside the states.
int check_written(const mhla_tensor_t* w, const mhla_tensor_t* const* others, int count, const float* const* states,
                  int n_states, int64_t bytes) {
  if (!non_overlapping(w)) return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (!disjoint(w, others[i])) return MHLA_ERR_INVALID_ARG;
  for (int i = 0; i < n_states; ++i)
    if (meets(w, states[i], bytes)) return MHLA_ERR_INVALID_ARG;
  return MHLA_OK;
}

bool states_aligned(std::initializer_list<const float*> ps) {
  for (const float* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return false;
  return true;
}

GatedProblem gated_problem(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                           const mhla_tensor_t* g, float scale) {
  GatedProblem p = {};
  p.B = q->B; p.N = q->N; p.H = q->H; p.d = static_cast<int32_t>(q->d);
  p.dtype = q->dtype;
  p.scale = scale;
  p.q = operand(q); p.k = operand(k); p.v = operand(v); p.g = operand(g);
  return p;
}

// Runs a launcher with the caller's workspace or a stream-ordered allocation.
template <typename Launch>
int with_workspace(size_t need, void* workspace, size_t workspace_bytes, void* stream, Launch launch) {
  void* ws = workspace;
  if (!ws && workspace_bytes != 0) return MHLA_ERR_WORKSPACE;
  if (ws && (workspace_bytes < need || reinterpret_cast<uintptr_t>(ws) % kAlign != 0)) return MHLA_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool owned = false;
  if (!ws && need > 0) {
    if (cudaMallocAsync(&ws, need, s) != cudaSuccess) return MHLA_ERR_CUDA;
    owned = true;
  }
  const int rc = launch(ws);
  if (owned && cudaFreeAsync(ws, s) != cudaSuccess && rc == MHLA_OK) return MHLA_ERR_CUDA;
  return rc;
}

}  // namespace
}  // namespace mhla

using namespace mhla;

// ----------------------------------------------------------------- recurrence

extern "C" mhla_status_t mhla_gated_workspace_size(const mhla_tensor_t* q, size_t* bytes) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const int rc = check_tensor(q);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  *bytes = empty(q) ? 0 : gated_workspace_bytes(gated_problem(q, q, q, q, 1.0f));
  return MHLA_OK;
}

extern "C" mhla_status_t mhla_gated_backward_workspace_size(const mhla_tensor_t* q, size_t* bytes) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const int rc = check_tensor(q);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  *bytes = empty(q) ? 0 : gated_bwd_workspace_bytes(gated_problem(q, q, q, q, 1.0f));
  return MHLA_OK;
}

extern "C" mhla_status_t mhla_gated_forward(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                            const mhla_tensor_t* g, float scale, const float* state_in,
                                            const mhla_tensor_t* out, float* state_out, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  int rc = check_gated(q, k, v, g, scale);
  if (rc == MHLA_OK) rc = check_elements(out);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(q, out)) return MHLA_ERR_SHAPE;
  if (empty(q)) return MHLA_OK;
  const mhla_tensor_t* in[] = {q, k, v, g};
  const float* states[] = {state_in, state_out};
  const int64_t sb = state_bytes(q);
  if (!states_aligned({state_in, state_out})) return MHLA_ERR_INVALID_ARG;
  rc = check_written(out, in, 4, states, 2, sb);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  for (const mhla_tensor_t* t : in)
    if (meets(t, state_out, sb)) return MHLA_ERR_INVALID_ARG;
  if (state_out != state_in && plain_overlap(state_in, state_out, sb)) return MHLA_ERR_INVALID_ARG;
  const GatedProblem p = gated_problem(q, k, v, g, scale);
  return static_cast<mhla_status_t>(
      with_workspace(gated_workspace_bytes(p), workspace, workspace_bytes, stream, [&](void* ws) {
        return launch_gated_forward(p, state_in, operand(out), state_out, ws, stream);
      }));
}

extern "C" mhla_status_t mhla_gated_backward(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                             const mhla_tensor_t* g, const mhla_tensor_t* dout, float scale,
                                             const float* state_in, const float* dstate_out, const mhla_tensor_t* dq,
                                             const mhla_tensor_t* dk, const mhla_tensor_t* dv,
                                             const mhla_tensor_t* dg, float* dstate_in, void* workspace,
                                             size_t workspace_bytes, void* stream) {
  int rc = check_gated(q, k, v, g, scale);
  for (const mhla_tensor_t* t : {dout, dq, dk, dv, dg})
    if (rc == MHLA_OK) rc = check_elements(t);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  for (const mhla_tensor_t* t : {dout, dq, dk, dv})
    if (!same_shape(q, t)) return MHLA_ERR_SHAPE;
  if (!gate_shape(q, dg)) return MHLA_ERR_SHAPE;
  if (empty(q)) return MHLA_OK;
  const mhla_tensor_t* all[] = {q, k, v, g, dout, dq, dk, dv, dg};
  const float* states[] = {state_in, dstate_out, dstate_in};
  const int64_t sb = state_bytes(q);
  if (!states_aligned({state_in, dstate_out, dstate_in})) return MHLA_ERR_INVALID_ARG;
  for (int i = 5; i < 9; ++i) {
    rc = check_written(all[i], all, i, states, 3, sb);
    if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  }
  for (int i = 0; i < 5; ++i)
    if (meets(all[i], dstate_in, sb)) return MHLA_ERR_INVALID_ARG;
  if (plain_overlap(dstate_in, state_in, sb) || plain_overlap(dstate_in, dstate_out, sb)) return MHLA_ERR_INVALID_ARG;
  const GatedProblem p = gated_problem(q, k, v, g, scale);
  const GatedBackward b = {operand(dout), operand(dq), operand(dk), operand(dv), operand(dg), state_in, dstate_out,
                           dstate_in};
  return static_cast<mhla_status_t>(
      with_workspace(gated_bwd_workspace_bytes(p), workspace, workspace_bytes, stream,
                     [&](void* ws) { return launch_gated_backward(p, b, ws, stream); }));
}

extern "C" mhla_status_t mhla_gated_step(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                         const mhla_tensor_t* g, float scale, float* state,
                                         const mhla_tensor_t* out, void* stream) {
  int rc = check_gated(q, k, v, g, scale);
  if (rc == MHLA_OK) rc = check_elements(out);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(q, out) || q->N != 1) return MHLA_ERR_SHAPE;
  if (empty(q)) return MHLA_OK;
  if (!state || !states_aligned({state})) return MHLA_ERR_INVALID_ARG;
  const mhla_tensor_t* in[] = {q, k, v, g};
  const float* states[] = {state};
  const int64_t sb = state_bytes(q);
  rc = check_written(out, in, 4, states, 1, sb);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  for (const mhla_tensor_t* t : in)
    if (meets(t, state, sb)) return MHLA_ERR_INVALID_ARG;
  return static_cast<mhla_status_t>(launch_gated_step(gated_problem(q, k, v, g, scale), state, operand(out), stream));
}

// ----------------------------------------------------------------- delta rule

namespace mhla {
namespace {

// [B, N, H, d] of the values beside [B, N, Hk, d] of the keys.
bool value_shape(const mhla_tensor_t* q, const mhla_tensor_t* v) {
  return q->B == v->B && q->N == v->N && q->d == v->d && q->dtype == v->dtype &&
         (q->H == 0 ? v->H == 0 : v->H % q->H == 0);
}

DeltaProblem delta_problem(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v, const mhla_tensor_t* g,
                           const mhla_tensor_t* beta, float scale) {
  DeltaProblem p = {};
  p.B = v->B; p.N = v->N; p.H = v->H; p.Hk = q->H; p.d = static_cast<int32_t>(v->d);
  p.dtype = v->dtype;
  p.scale = scale;
  p.q = operand(q); p.k = operand(k); p.v = operand(v); p.g = operand(g); p.beta = operand(beta);
  return p;
}

// Each CTA owns a chunk of a (b, h): their number fits a 31-bit grid axis.
bool delta_fits(const mhla_tensor_t* v) {
  const int64_t heads = v->B > (int64_t{1} << 24) || v->H > (int64_t{1} << 24) ? int64_t{1} << 25 : v->B * v->H;
  return heads <= (int64_t{1} << 24) && v->N <= (int64_t{1} << 36) &&
         heads * ((v->N + 31) / 32) < (int64_t{1} << 31);   // the shorter of both types' chunks
}

int check_delta(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v, const mhla_tensor_t* g,
                const mhla_tensor_t* beta, float scale) {
  for (const mhla_tensor_t* t : {q, k, v, g, beta}) {
    const int rc = check_elements(t);
    if (rc != MHLA_OK) return rc;
  }
  if (!same_shape(q, k) || !value_shape(q, v) || !gate_shape(v, g) || !gate_shape(v, beta)) return MHLA_ERR_SHAPE;
  if (!std::isfinite(scale)) return MHLA_ERR_INVALID_ARG;
  return delta_fits(v) ? MHLA_OK : MHLA_ERR_UNSUPPORTED;
}

template <typename Bytes>
int delta_size(const mhla_tensor_t* q, const mhla_tensor_t* v, size_t* bytes, Bytes need) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  for (const mhla_tensor_t* t : {q, v}) {
    const int rc = check_tensor(t);
    if (rc != MHLA_OK) return rc;
  }
  if (!value_shape(q, v)) return MHLA_ERR_SHAPE;
  if (!delta_fits(v)) return MHLA_ERR_UNSUPPORTED;
  *bytes = empty(v) ? 0 : need(delta_problem(q, q, v, v, v, 1.0f));
  return MHLA_OK;
}

}  // namespace
}  // namespace mhla

extern "C" mhla_status_t mhla_delta_workspace_size(const mhla_tensor_t* q, const mhla_tensor_t* v, size_t* bytes) {
  return static_cast<mhla_status_t>(delta_size(q, v, bytes, delta_workspace_bytes));
}

extern "C" mhla_status_t mhla_delta_backward_workspace_size(const mhla_tensor_t* q, const mhla_tensor_t* v, size_t* bytes) {
  return static_cast<mhla_status_t>(delta_size(q, v, bytes, delta_bwd_workspace_bytes));
}

extern "C" mhla_status_t mhla_delta_forward(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                            const mhla_tensor_t* g, const mhla_tensor_t* beta, float scale,
                                            const float* state_in, const mhla_tensor_t* out, float* state_out,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_delta(q, k, v, g, beta, scale);
  if (rc == MHLA_OK) rc = check_elements(out);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(v, out)) return MHLA_ERR_SHAPE;
  if (empty(v)) return MHLA_OK;
  const mhla_tensor_t* in[] = {q, k, v, g, beta};
  const float* states[] = {state_in, state_out};
  const int64_t sb = state_bytes(v);
  if (!states_aligned({state_in, state_out})) return MHLA_ERR_INVALID_ARG;
  rc = check_written(out, in, 5, states, 2, sb);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  for (const mhla_tensor_t* t : in)
    if (meets(t, state_out, sb)) return MHLA_ERR_INVALID_ARG;
  if (state_out != state_in && plain_overlap(state_in, state_out, sb)) return MHLA_ERR_INVALID_ARG;
  const DeltaProblem p = delta_problem(q, k, v, g, beta, scale);
  return static_cast<mhla_status_t>(
      with_workspace(delta_workspace_bytes(p), workspace, workspace_bytes, stream, [&](void* ws) {
        return launch_delta_forward(p, state_in, operand(out), state_out, ws, stream);
      }));
}

extern "C" mhla_status_t mhla_delta_backward(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                             const mhla_tensor_t* g, const mhla_tensor_t* beta, const mhla_tensor_t* dout,
                                             float scale, const float* state_in, const float* dstate_out,
                                             const mhla_tensor_t* dq, const mhla_tensor_t* dk, const mhla_tensor_t* dv,
                                             const mhla_tensor_t* dg, const mhla_tensor_t* dbeta, float* dstate_in,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_delta(q, k, v, g, beta, scale);
  for (const mhla_tensor_t* t : {dout, dq, dk, dv, dg, dbeta})
    if (rc == MHLA_OK) rc = check_elements(t);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(v, dout) || !same_shape(v, dv) || !same_shape(q, dq) || !same_shape(q, dk) || !gate_shape(v, dg) ||
      !gate_shape(v, dbeta))
    return MHLA_ERR_SHAPE;
  if (v->H == 0 && !empty(q)) return MHLA_ERR_SHAPE;   // nothing would write the elements of dq and dk
  if (empty(v)) return MHLA_OK;
  const mhla_tensor_t* all[] = {q, k, v, g, beta, dout, dq, dk, dv, dg, dbeta};
  constexpr int kInputs = 6, kAll = 11;
  const float* states[] = {state_in, dstate_out, dstate_in};
  const int64_t sb = state_bytes(v);
  if (!states_aligned({state_in, dstate_out, dstate_in})) return MHLA_ERR_INVALID_ARG;
  for (int i = kInputs; i < kAll; ++i) {
    rc = check_written(all[i], all, i, states, 3, sb);
    if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  }
  for (int i = 0; i < kInputs; ++i)
    if (meets(all[i], dstate_in, sb)) return MHLA_ERR_INVALID_ARG;
  if (plain_overlap(dstate_in, state_in, sb) || plain_overlap(dstate_in, dstate_out, sb)) return MHLA_ERR_INVALID_ARG;
  const DeltaProblem p = delta_problem(q, k, v, g, beta, scale);
  const DeltaBackward b = {operand(dout), operand(dq), operand(dk), operand(dv), operand(dg), operand(dbeta), state_in,
                           dstate_out, dstate_in};
  return static_cast<mhla_status_t>(
      with_workspace(delta_bwd_workspace_bytes(p), workspace, workspace_bytes, stream,
                     [&](void* ws) { return launch_delta_backward(p, b, ws, stream); }));
}

extern "C" mhla_status_t mhla_delta_step(const mhla_tensor_t* q, const mhla_tensor_t* k, const mhla_tensor_t* v,
                                         const mhla_tensor_t* g, const mhla_tensor_t* beta, float scale, float* state,
                                         const mhla_tensor_t* out, void* stream) {
  int rc = check_delta(q, k, v, g, beta, scale);
  if (rc == MHLA_OK) rc = check_elements(out);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(v, out) || v->N != 1) return MHLA_ERR_SHAPE;
  if (empty(v)) return MHLA_OK;
  if (!state || !states_aligned({state})) return MHLA_ERR_INVALID_ARG;
  const mhla_tensor_t* in[] = {q, k, v, g, beta};
  const float* states[] = {state};
  const int64_t sb = state_bytes(v);
  rc = check_written(out, in, 5, states, 1, sb);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  for (const mhla_tensor_t* t : in)
    if (meets(t, state, sb)) return MHLA_ERR_INVALID_ARG;
  return static_cast<mhla_status_t>(launch_delta_step(delta_problem(q, k, v, g, beta, scale), state, operand(out), stream));
}

// ----------------------------------------------------------------- norm and rotation

namespace mhla {
namespace {

int qk_norm_problem(const mhla_tensor_t* q, const mhla_tensor_t* k, const float* q_weight, const float* k_weight,
                    float eps, const mhla_rotation_t* rot, QkNormProblem* p) {
  for (const mhla_tensor_t* t : {q, k}) {
    const int rc = check_elements(t);
    if (rc != MHLA_OK) return rc;
  }
  if (q->B != k->B || q->N != k->N || q->d != k->d || q->dtype != k->dtype) return MHLA_ERR_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return MHLA_ERR_INVALID_ARG;
  if (q->B > (int64_t{1} << 31) || q->N > (int64_t{1} << 40) || q->H > (int64_t{1} << 20) ||
      k->H > (int64_t{1} << 20) || q->B * q->N > (int64_t{1} << 40))
    return MHLA_ERR_UNSUPPORTED;
  if (!states_aligned({q_weight, k_weight})) return MHLA_ERR_INVALID_ARG;
  QkNormProblem& P = *p;
  P = {};
  P.B = q->B; P.N = q->N; P.Hq = q->H; P.Hk = k->H; P.d = static_cast<int32_t>(q->d);
  P.dtype = q->dtype;
  P.eps = eps;
  P.q = operand(q); P.k = operand(k);
  P.q_weight = q_weight; P.k_weight = k_weight;
  if (rot && rot->table) {
    if (rot->layout != MHLA_ROTATION_HALF && rot->layout != MHLA_ROTATION_INTERLEAVED) return MHLA_ERR_INVALID_ARG;
    if (rot->pairs < 0 || rot->rows < 0) return MHLA_ERR_INVALID_ARG;
    if (rot->rows > (int64_t{1} << 40)) return MHLA_ERR_UNSUPPORTED;   // their bytes fit 64 bits below
    if (reinterpret_cast<uintptr_t>(rot->table) % 8 != 0 || reinterpret_cast<uintptr_t>(rot->positions) % 4 != 0)
      return MHLA_ERR_INVALID_ARG;
    if (2 * static_cast<int64_t>(rot->pairs) > q->d) return MHLA_ERR_SHAPE;
    if (!rot->positions && rot->rows < q->N) return MHLA_ERR_SHAPE;
    P.table = rot->table;
    P.positions = rot->positions;
    P.rows = rot->rows;
    P.pairs = rot->pairs;
    P.interleaved = rot->layout == MHLA_ROTATION_INTERLEAVED;
  }
  if (P.pairs == 0) {
    P.table = nullptr;
    P.positions = nullptr;
  }
  return MHLA_OK;
}

// out shares no element with the tensors given (out == twin in address and
// strides is fine), nor with the plain memory the call reads.
int check_normed(const QkNormProblem& p, const mhla_tensor_t* out, const mhla_tensor_t* twin,
                 std::initializer_list<const mhla_tensor_t*> others) {
  if (empty(out)) return MHLA_OK;
  if (!non_overlapping(out)) return MHLA_ERR_INVALID_ARG;
  if (!same_view(out, twin) && !disjoint(out, twin)) return MHLA_ERR_INVALID_ARG;
  for (const mhla_tensor_t* t : others)
    if (!empty(t) && !disjoint(out, t)) return MHLA_ERR_INVALID_ARG;
  if (meets(out, p.q_weight, 4 * p.d) || meets(out, p.k_weight, 4 * p.d) ||
      meets(out, p.table, p.rows * p.pairs * 8) || meets(out, p.positions, p.B * p.N * 4))
    return MHLA_ERR_INVALID_ARG;
  return MHLA_OK;
}

}  // namespace
}  // namespace mhla

extern "C" mhla_status_t mhla_qk_norm(const mhla_tensor_t* q, const mhla_tensor_t* k, const float* q_weight,
                                      const float* k_weight, float eps, const mhla_rotation_t* rot,
                                      const mhla_tensor_t* q_out, const mhla_tensor_t* k_out, void* stream) {
  QkNormProblem p;
  int rc = qk_norm_problem(q, k, q_weight, k_weight, eps, rot, &p);
  for (const mhla_tensor_t* t : {q_out, k_out})
    if (rc == MHLA_OK) rc = check_elements(t);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(q, q_out) || !same_shape(k, k_out)) return MHLA_ERR_SHAPE;
  rc = check_normed(p, q_out, q, {k, k_out});
  if (rc == MHLA_OK) rc = check_normed(p, k_out, k, {q});
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (p.B == 0 || (p.Hq == 0 && p.Hk == 0)) return MHLA_OK;
  p.q_out = operand(q_out);
  p.k_out = operand(k_out);
  return static_cast<mhla_status_t>(launch_qk_norm(p, stream));
}

extern "C" mhla_status_t mhla_qk_norm_backward_workspace_size(const mhla_tensor_t* q, size_t* bytes) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const int rc = check_tensor(q);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  *bytes = qk_norm_bwd_workspace_bytes(static_cast<int32_t>(q->d));
  return MHLA_OK;
}

extern "C" mhla_status_t mhla_qk_norm_backward(const mhla_tensor_t* q, const mhla_tensor_t* k, const float* q_weight,
                                               const float* k_weight, float eps, const mhla_rotation_t* rot,
                                               const mhla_tensor_t* dq_out, const mhla_tensor_t* dk_out,
                                               const mhla_tensor_t* dq, const mhla_tensor_t* dk, float* dq_weight,
                                               float* dk_weight, void* workspace, size_t workspace_bytes,
                                               void* stream) {
  QkNormProblem p;
  int rc = qk_norm_problem(q, k, q_weight, k_weight, eps, rot, &p);
  for (const mhla_tensor_t* t : {dq_out, dk_out, dq, dk})
    if (rc == MHLA_OK) rc = check_elements(t);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!same_shape(q, dq_out) || !same_shape(k, dk_out) || !same_shape(q, dq) || !same_shape(k, dk))
    return MHLA_ERR_SHAPE;
  rc = check_normed(p, dq, dq_out, {q, k, dk_out, dk});
  if (rc == MHLA_OK) rc = check_normed(p, dk, dk_out, {q, k, dq_out});
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (!states_aligned({dq_weight, dk_weight}) || plain_overlap(dq_weight, dk_weight, 4 * p.d))
    return MHLA_ERR_INVALID_ARG;
  for (const float* w : {dq_weight, dk_weight}) {
    if (plain_overlap(w, q_weight, 4 * p.d) || plain_overlap(w, k_weight, 4 * p.d) ||
        plain_overlap(w, p.table, 4 * p.d, p.rows * p.pairs * 8) || plain_overlap(w, p.positions, 4 * p.d, p.B * p.N * 4))
      return MHLA_ERR_INVALID_ARG;
    for (const mhla_tensor_t* t : {q, k, dq_out, dk_out, dq, dk})
      if (!empty(t) && meets(t, w, 4 * p.d)) return MHLA_ERR_INVALID_ARG;
  }
  p.dq_out = operand(dq_out);
  p.dk_out = operand(dk_out);
  p.q_out = operand(dq);
  p.k_out = operand(dk);
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  return static_cast<mhla_status_t>(with_workspace(qk_norm_bwd_workspace_bytes(p.d), workspace, workspace_bytes,
                                                   stream,
                                                   [&](void* ws) { return launch_qk_norm_backward(p, ws, stream); }));
}

// ----------------------------------------------------------------- linear layer

namespace mhla {
namespace {

int check_linear(int64_t rows, int64_t k, int64_t n, int32_t dtype, int32_t act) {
  if (rows < 0 || k < 1 || n < 1 || !valid_dtype(dtype) || act < MHLA_ACT_NONE || act > MHLA_ACT_SILU) return MHLA_ERR_INVALID_ARG;
  if (rows >= (int64_t{1} << 31) || k > (int64_t{1} << 20) || n > (int64_t{1} << 20)) return MHLA_ERR_UNSUPPORTED;
  return MHLA_OK;
}

struct Block {
  const void* p;
  int64_t bytes;
};
bool apart(const Block& w, std::initializer_list<Block> others) {
  for (const Block& o : others)
    if (plain_overlap(w.p, o.p, w.bytes, o.bytes)) return false;
  return true;
}
bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

}  // namespace
}  // namespace mhla

extern "C" mhla_status_t mhla_linear_act_workspace_size(int64_t rows, int64_t k, int64_t n, int32_t dtype, size_t* bytes) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const int rc = check_linear(rows, k, n, dtype, MHLA_ACT_NONE);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  *bytes = rows == 0 ? 0 : linear_act_workspace_bytes(LinearProblem{nullptr, nullptr, rows, k, n, dtype, MHLA_ACT_NONE});
  return MHLA_OK;
}

extern "C" mhla_status_t mhla_linear_act_backward_workspace_size(int64_t rows, int64_t k, int64_t n, int32_t dtype,
                                                                 int32_t activation, size_t* bytes) {
  if (!bytes) return MHLA_ERR_INVALID_ARG;
  const int rc = check_linear(rows, k, n, dtype, activation);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  *bytes = rows == 0 ? 0 : linear_act_bwd_workspace_bytes(LinearProblem{nullptr, nullptr, rows, k, n, dtype, activation});
  return MHLA_OK;
}

extern "C" mhla_status_t mhla_linear_act(const void* x, const void* w, const void* bias, int32_t activation,
                                         const void* residual, void* pre, void* out, int64_t rows, int64_t k, int64_t n,
                                         int32_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_linear(rows, k, n, dtype, activation);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (rows == 0) return MHLA_OK;
  if (!x || !w || !out || !all_aligned({x, w, bias, residual, pre, out})) return MHLA_ERR_INVALID_ARG;
  const int64_t e = elem_bytes(dtype);
  const Block o = {out, rows * n * e}, z = {pre, rows * n * e};
  const Block bx = {x, rows * k * e}, bw = {w, n * k * e}, bb = {bias, n * e}, br = {residual, rows * n * e};
  if (!apart(o, {z, bx, bw, bb}) || (residual != out && !apart(o, {br})) || !apart(z, {bx, bw, bb, br})) return MHLA_ERR_INVALID_ARG;
  const LinearProblem p = {x, w, rows, k, n, dtype, activation};
  return static_cast<mhla_status_t>(
      with_workspace(linear_act_workspace_bytes(p), workspace, workspace_bytes, stream,
                     [&](void* ws) { return launch_linear_act(p, bias, residual, pre, out, ws, stream); }));
}

extern "C" mhla_status_t mhla_linear_act_backward(const void* x, const void* w, const void* dout, const void* pre,
                                                  int32_t activation, void* dx, void* dw, void* dbias, int64_t rows, int64_t k,
                                                  int64_t n, int32_t dtype, void* workspace, size_t workspace_bytes,
                                                  void* stream) {
  const int rc = check_linear(rows, k, n, dtype, activation);
  if (rc != MHLA_OK) return static_cast<mhla_status_t>(rc);
  if (activation == MHLA_ACT_NONE) pre = nullptr;   // unused, whatever it is
  if (!all_aligned({x, w, dout, pre, dx, dw, dbias})) return MHLA_ERR_INVALID_ARG;
  const int64_t e = elem_bytes(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(n * k * e), s) != cudaSuccess) return MHLA_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(n * e), s) != cudaSuccess) return MHLA_ERR_CUDA;
    return MHLA_OK;
  }
  if (!x || !w || !dout || (activation != MHLA_ACT_NONE && !pre)) return MHLA_ERR_INVALID_ARG;
  const Block in[] = {{x, rows * k * e}, {w, n * k * e}, {dout, rows * n * e}, {pre, rows * n * e}};
  const Block bx = {dx, rows * k * e}, bw = {dw, n * k * e}, bb = {dbias, n * e};
  for (const Block& o : {bx, bw, bb})
    if (!apart(o, {in[0], in[1], in[2], in[3]})) return MHLA_ERR_INVALID_ARG;
  if (!apart(bx, {bw, bb}) || !apart(bw, {bb})) return MHLA_ERR_INVALID_ARG;
  if (!dx && !dw && !dbias) return MHLA_OK;
  const LinearProblem p = {x, w, rows, k, n, dtype, activation};
  return static_cast<mhla_status_t>(
      with_workspace(linear_act_bwd_workspace_bytes(p), workspace, workspace_bytes, stream,
                     [&](void* ws) { return launch_linear_act_backward(p, dout, pre, dx, dw, dbias, ws, stream); }));
}
