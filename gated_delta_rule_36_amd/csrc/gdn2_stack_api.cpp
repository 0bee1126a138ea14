// C ABI of what stands around the mixer in a stack (diagonal recurrence, norm between layers,
// verification of drafts): argument validation, launch. Declarations and the contract of every
// entry point are in include/gdn2.h.
#include "../../include/gdn2.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "gdn2_stack_launch.h"

namespace {

bool aligned(const void* p, unsigned a) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
bool all_aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return false;
  return true;
}
bool dtype_ok(int dtype) { return dtype == GDN2_BF16 || dtype == GDN2_F32; }
bool stride_ok(int64_t stride, int D) { return stride >= D && stride % 8 == 0; }
// (the recurrence's kernels keep a tile's offsets in 32 bits)
bool token_stride_ok(int64_t stride, int D) { return stride_ok(stride, D) && stride <= gdn2::kMaxStride; }
int status_of(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_LAUNCH_FAILED; }

// Sizes, strides and inputs that the whole-sequence forward and backward share.
int check_recurrence(bool backward, const void* v, const void* g, const void* w, const int32_t* cu_seqlens, int B,
                     int T, int D, int N, int64_t v_stride, int64_t g_stride, int64_t w_stride,
                     int dtype) {
  if (!dtype_ok(dtype) || B < 0 || T < 0 || D <= 0 || N < 0) return GDN2_INVALID_ARGUMENT;
  if (cu_seqlens == nullptr ? N != B : B != 1) return GDN2_INVALID_ARGUMENT;
  if (D % 8 != 0) return GDN2_UNSUPPORTED;
  if (!token_stride_ok(v_stride, D) || !token_stride_ok(g_stride, D) ||
      (w != nullptr && !token_stride_ok(w_stride, D)))
    return GDN2_INVALID_ARGUMENT;
  if ((long)B * T > (long)INT_MAX - 4096) return GDN2_INVALID_ARGUMENT;
  if (gdn2::recurrence_groups(gdn2::recurrence_cut(backward, cu_seqlens != nullptr, B, T, D, N), D) > gdn2::kMaxGroups)
    return GDN2_INVALID_ARGUMENT;
  if ((long)B * T > 0 && (!v || !g)) return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({v, g, w}) || !aligned(cu_seqlens, 4)) return GDN2_INVALID_ARGUMENT;
  return GDN2_OK;
}

gdn2::RecurrenceArgs recurrence_args(bool backward, const void* v, const void* g, const void* w,
                                     const int32_t* cu_seqlens, int B, int T, int D, int N,
                                     int64_t v_stride, int64_t g_stride, int64_t w_stride,
                                     int dtype, void* workspace, void* stream) {
  gdn2::RecurrenceArgs a{};
  a.v = v; a.g = g; a.w = w; a.cu_seqlens = cu_seqlens;
  a.v_stride = v_stride; a.g_stride = g_stride; a.w_stride = w_stride;
  a.T = T; a.N = N; a.D = D; a.dtype = dtype; a.stream = stream;
  a.cut = gdn2::recurrence_cut(backward, cu_seqlens != nullptr, B, T, D, N);
  a.cut.maps = static_cast<float*>(workspace);
  return a;
}

// Width, types and strides of the norm.
int check_norm(int64_t rows, int D, float eps, int dtype, int r_dtype) {
  if (!dtype_ok(dtype) || !dtype_ok(r_dtype) || rows < 0 || D <= 0) return GDN2_INVALID_ARGUMENT;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return GDN2_INVALID_ARGUMENT;
  if (D % 8 != 0 || D > gdn2::kNormMaxWidth) return GDN2_UNSUPPORTED;
  if (dtype == GDN2_F32 && r_dtype != GDN2_F32) return GDN2_UNSUPPORTED;
  if (rows > gdn2::kMaxGroups) return GDN2_INVALID_ARGUMENT;
  return GDN2_OK;
}

}  // namespace

extern "C" {

size_t gdn2_linear_recurrence_workspace_bytes(int backward, int packed, int B, int T, int D, int N) {
  if (B < 0 || T < 0 || D <= 0 || D % 8 != 0 || N < 0 || (packed ? B != 1 : N != B) ||
      (long)B * T > (long)INT_MAX - 4096)
    return 0;
  return gdn2::recurrence_workspace_bytes(gdn2::recurrence_cut(backward != 0, packed != 0, B, T, D, N), D);
}

size_t gdn2_linear_recurrence_states_bytes(int packed, int B, int T, int D, int N) {
  if (B < 0 || T < 0 || D <= 0 || D % 8 != 0 || N < 0 || (packed ? B != 1 : N != B)) return 0;
  return (size_t)gdn2::recurrence_state_slots(packed != 0, B, T, N) * D * sizeof(float);
}

int gdn2_linear_recurrence(const void* v, const void* log_alpha, const void* w,
                           const float* initial_state, void* o, float* final_state, float* states,
                           const int32_t* cu_seqlens, int B, int T, int D, int N,
                           int64_t v_stride, int64_t g_stride, int64_t w_stride, int dtype,
                           void* workspace, size_t workspace_bytes, void* hip_stream) {
  const int st = check_recurrence(false, v, log_alpha, w, cu_seqlens, B, T, D, N, v_stride, g_stride,
                                  w_stride, dtype);
  if (st != GDN2_OK) return st;
  if ((long)B * T > 0 && !o && !states) return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({initial_state, o, final_state, states, workspace})) return GDN2_INVALID_ARGUMENT;
  // (the training forward writes the rows of no sequence)
  if (N == 0 && !(cu_seqlens && T > 0 && states && o)) return GDN2_OK;
  const size_t need = gdn2_linear_recurrence_workspace_bytes(0, cu_seqlens != nullptr, B, T, D, N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN2_WORKSPACE_TOO_SMALL;
  gdn2::RecurrenceArgs a = recurrence_args(false, v, log_alpha, w, cu_seqlens, B, T, D, N, v_stride,
                                           g_stride, w_stride, dtype, workspace, hip_stream);
  a.s0 = initial_state; a.o = o; a.sN = final_state; a.states = states;
  // (of two passes only the first reads the initial states, and a sequence of several units gets its final
  // one in the second)
  if (final_state != nullptr && final_state == initial_state) a.cut.twice = true;
  return status_of(gdn2::launch_recurrence(a));
}

int gdn2_linear_recurrence_bwd(const void* v, const void* log_alpha, const void* w,
                               const float* states, const void* d_o, const float* d_final_state,
                               void* dv, void* dlog_alpha, void* dw, float* d_initial_state,
                               const int32_t* cu_seqlens, int B, int T, int D, int N,
                               int64_t v_stride, int64_t g_stride, int64_t w_stride, int dtype,
                               void* workspace, size_t workspace_bytes, void* hip_stream) {
  const int st = check_recurrence(true, v, log_alpha, w, cu_seqlens, B, T, D, N, v_stride, g_stride,
                                  w_stride, dtype);
  if (st != GDN2_OK) return st;
  if ((long)B * T > 0 && (!states || !d_o || !dv || !dlog_alpha || (w != nullptr && !dw)))
    return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({states, d_o, d_final_state, dv, dlog_alpha, dw, d_initial_state,
                      workspace}))
    return GDN2_INVALID_ARGUMENT;
  if (N == 0 && (long)B * T == 0) return GDN2_OK;
  const size_t need = gdn2_linear_recurrence_workspace_bytes(1, cu_seqlens != nullptr, B, T, D, N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN2_WORKSPACE_TOO_SMALL;
  gdn2::RecurrenceBwdArgs b{};
  b.f = recurrence_args(true, v, log_alpha, w, cu_seqlens, B, T, D, N, v_stride, g_stride, w_stride,
                        dtype, workspace, hip_stream);
  b.f.states = const_cast<float*>(states);
  b.d_o = d_o; b.d_sN = d_final_state;
  b.dv = dv; b.dg = dlog_alpha; b.dw = dw; b.d_s0 = d_initial_state;
  return status_of(gdn2::launch_recurrence_bwd(b));
}

int gdn2_linear_recurrence_tokens(const void* v, const void* log_alpha, const void* w,
                                  float* state_pool, const int32_t* state_indices,
                                  const int32_t* commit_len, void* o, float* step_states, int N,
                                  int L, int D, int P, int64_t v_stride, int64_t g_stride,
                                  int64_t w_stride, int dtype, void* hip_stream) {
  if (!dtype_ok(dtype) || N < 0 || L < 0 || D <= 0 || P < 0) return GDN2_INVALID_ARGUMENT;
  if (D % 8 != 0) return GDN2_UNSUPPORTED;
  if (!token_stride_ok(v_stride, D) || !token_stride_ok(g_stride, D) ||
      (w != nullptr && !token_stride_ok(w_stride, D)))
    return GDN2_INVALID_ARGUMENT;
  if (N == 0 || L == 0) return GDN2_OK;
  if (!v || !log_alpha || !state_pool || !o) return GDN2_INVALID_ARGUMENT;
  if (state_indices == nullptr && P < N) return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({v, log_alpha, w, state_pool, o, step_states}) || !aligned(state_indices, 4) ||
      !aligned(commit_len, 4))
    return GDN2_INVALID_ARGUMENT;
  if ((long)N * L > (long)INT_MAX || (long)N * (D / 8) > (long)INT_MAX) return GDN2_INVALID_ARGUMENT;
  gdn2::RecurrenceTokensArgs a{};
  a.v = v; a.g = log_alpha; a.w = w; a.pool = state_pool; a.indices = state_indices;
  a.commit = commit_len; a.o = o; a.step_states = step_states;
  a.v_stride = v_stride; a.g_stride = g_stride; a.w_stride = w_stride;
  a.N = N; a.L = L; a.D = D; a.P = P; a.dtype = dtype; a.stream = hip_stream;
  return status_of(gdn2::launch_recurrence_tokens(a));
}

int gdn2_residual_norm(const void* x, const void* residual, const float* weight, void* y, void* h,
                       float* scale, int64_t rows, int D, int64_t x_stride, int64_t r_stride,
                       int group, float eps, int dtype, int r_dtype, void* hip_stream) {
  const int st = check_norm(rows, D, eps, dtype, r_dtype);
  if (st != GDN2_OK) return st;
  if (group < 0) return GDN2_INVALID_ARGUMENT;
  if (group != 0 && group != 32 && group != 64 && group != 128) return GDN2_UNSUPPORTED;
  if (group != 0 && D % group != 0) return GDN2_INVALID_ARGUMENT;
  if (!stride_ok(x_stride, D) || (residual != nullptr && !stride_ok(r_stride, D)))
    return GDN2_INVALID_ARGUMENT;
  if (residual == nullptr && r_dtype != dtype) return GDN2_INVALID_ARGUMENT;
  if (rows == 0) return GDN2_OK;
  if (!x || !weight || !y || (residual != nullptr && !h) || (scale == nullptr && group != 0))
    return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({x, residual, weight, y, h}) || !aligned(scale, 4)) return GDN2_INVALID_ARGUMENT;
  gdn2::ResidualNormArgs a{};
  a.x = x; a.r = residual; a.weight = weight; a.y = y; a.h = h; a.scale = scale;
  a.rows = rows; a.x_stride = x_stride; a.r_stride = r_stride;
  a.D = D; a.group = group == 0 ? D : group; a.eps = eps;
  a.dtype = dtype; a.r_dtype = r_dtype; a.stream = hip_stream;
  return status_of(gdn2::launch_residual_norm(a));
}

size_t gdn2_residual_norm_bwd_workspace_bytes(int64_t rows, int D) {
  if (rows <= 0 || D <= 0 || D % 8 != 0 || D > gdn2::kNormMaxWidth || rows > gdn2::kMaxGroups) return 0;
  return (size_t)gdn2::residual_norm_bwd_groups(rows, D) * D * sizeof(float);
}

int gdn2_residual_norm_bwd(const void* dy, const void* dh, const void* h, const float* weight,
                           void* dx, void* dr, float* dweight, int64_t rows, int D,
                           int64_t h_stride, float eps, int dtype, int r_dtype, void* workspace,
                           size_t workspace_bytes, void* hip_stream) {
  const int st = check_norm(rows, D, eps, dtype, r_dtype);
  if (st != GDN2_OK) return st;
  if (!stride_ok(h_stride, D) || (dtype == r_dtype) != (dr == nullptr)) return GDN2_INVALID_ARGUMENT;
  if (rows == 0) return GDN2_OK;
  if (!dy || !h || !weight || !dx || !dweight) return GDN2_INVALID_ARGUMENT;
  if (!all_aligned16({dy, dh, h, weight, dx, dr, dweight, workspace})) return GDN2_INVALID_ARGUMENT;
  if (workspace == nullptr || workspace_bytes < gdn2_residual_norm_bwd_workspace_bytes(rows, D))
    return GDN2_WORKSPACE_TOO_SMALL;
  gdn2::ResidualNormBwdArgs a{};
  a.dy = dy; a.dh = dh; a.h = h; a.weight = weight; a.dx = dx; a.dr = dr; a.dweight = dweight;
  a.partial = static_cast<float*>(workspace);
  a.rows = rows; a.h_stride = h_stride; a.D = D; a.eps = eps;
  a.dtype = dtype; a.r_dtype = r_dtype; a.stream = hip_stream;
  return status_of(gdn2::launch_residual_norm_bwd(a));
}

size_t gdn2_verify_drafts_workspace_bytes(int N, int V) {
  if (N <= 0 || V <= 0) return 0;
  return (size_t)N * gdn2::verify_pieces(V) * 2 * sizeof(double);
}

int gdn2_verify_drafts(const void* target_probs, const void* draft_probs, const int32_t* drafts,
                       const int32_t* draft_len, const float* uniforms, int32_t* tokens,
                       int32_t* commit_len, int N, int L, int V, int dtype, void* workspace,
                       size_t workspace_bytes, void* hip_stream) {
  if (!dtype_ok(dtype) || N < 0 || L < 0 || V <= 0) return GDN2_INVALID_ARGUMENT;
  if (L > (1 << 20) || V > (1 << 28)) return GDN2_INVALID_ARGUMENT;
  if (N == 0) return GDN2_OK;
  if (!target_probs || !uniforms || !tokens || !commit_len || (L > 0 && !drafts))
    return GDN2_INVALID_ARGUMENT;
  const unsigned size = dtype == GDN2_F32 ? 4 : 2;
  if (!aligned(target_probs, size) || !aligned(draft_probs, size) || !aligned(drafts, 4) ||
      !aligned(draft_len, 4) || !aligned(uniforms, 4) || !aligned(tokens, 4) ||
      !aligned(commit_len, 4) || !aligned(workspace, 16))
    return GDN2_INVALID_ARGUMENT;
  if ((long)N * gdn2::verify_pieces(V) > gdn2::kMaxGroups) return GDN2_INVALID_ARGUMENT;
  if (workspace == nullptr || workspace_bytes < gdn2_verify_drafts_workspace_bytes(N, V))
    return GDN2_WORKSPACE_TOO_SMALL;
  gdn2::VerifyArgs a{};
  a.p = target_probs; a.q = L > 0 ? draft_probs : nullptr; a.drafts = drafts;
  a.draft_len = draft_len; a.u = uniforms; a.tokens = tokens; a.commit = commit_len;
  a.sums = static_cast<double*>(workspace);
  a.N = N; a.L = L; a.V = V; a.dtype = dtype; a.stream = hip_stream;
  return status_of(gdn2::launch_verify(a));
}

}  // extern "C"
