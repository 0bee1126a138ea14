// C ABI of the softmax-attention layer: argument validation, launch. Declarations and the
// contract of every entry point are in include/gdn2.h.
#include "../../include/gdn2.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "gdn2_attn_launch.h"

namespace {

bool aligned(const void* p, unsigned a) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
bool width_ok(int d) { return d == 64 || d == 128; }
int status_of(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_LAUNCH_FAILED; }

constexpr int kRopeMask = GDN2_ROPE_INTERLEAVED | GDN2_ROPE_NO_NORM;

// Rotation, norm and row arguments that all three row entry points share.
int check_rows(int Hq, int Hk, int d, int rot, float eps, int flags, int dtype, const float* inv_freq,
               const float* q_weight, const float* k_weight) {
  if (dtype != GDN2_BF16 && dtype != GDN2_F32) return GDN2_INVALID_ARGUMENT;
  if ((flags & ~kRopeMask) != 0 || Hq <= 0 || Hk <= 0 || d <= 0) return GDN2_INVALID_ARGUMENT;
  if (!width_ok(d)) return GDN2_UNSUPPORTED;
  if (rot < 0 || rot > d || rot % 8 != 0) return GDN2_INVALID_ARGUMENT;
  if (rot > 0 && inv_freq == nullptr) return GDN2_INVALID_ARGUMENT;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return GDN2_INVALID_ARGUMENT;
  if (!aligned(inv_freq, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return GDN2_INVALID_ARGUMENT;
  if (Hq > (1 << 16) || Hk > (1 << 16)) return GDN2_INVALID_ARGUMENT;  // grid's second axis
  return GDN2_OK;
}

bool stride_ok(long stride, int H, int d) { return stride >= (long)H * d && stride % 8 == 0; }

// Cache, table and sequence arguments of the two serving entry points.
int check_cache(const void* k_cache, const void* v_cache, const float* k_scale,
                const float* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                const int32_t* cu_seqlens, int B, int T, int Hq, int Hk, int d, int N, int P,
                int max_blocks, int dtype) {
  if (dtype != GDN2_BF16 && dtype != GDN2_F32) return GDN2_INVALID_ARGUMENT;
  if (B < 0 || T < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0 || d <= 0 || N < 0 || P < 0 ||
      max_blocks < 0)
    return GDN2_INVALID_ARGUMENT;
  if (cu_seqlens == nullptr ? N != B : B != 1) return GDN2_INVALID_ARGUMENT;
  if (!width_ok(d) || dtype != GDN2_BF16) return GDN2_UNSUPPORTED;
  if (N == 0 || T == 0) return GDN2_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens)
    return GDN2_INVALID_ARGUMENT;
  if (P == 0 || max_blocks == 0) return GDN2_INVALID_ARGUMENT;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_seqlens, 4))
    return GDN2_INVALID_ARGUMENT;
  if ((long)B * T > (long)INT_MAX || (long)max_blocks * gdn2::kCacheBlock > (long)INT_MAX)
    return GDN2_INVALID_ARGUMENT;
  return GDN2_OK;
}

gdn2::CacheView view(const void* k_cache, const void* v_cache, const float* k_scale,
                     const float* v_scale, const int32_t* block_table, const int32_t* seq_lens,
                     const int32_t* cu_seqlens, int T, int N, int P, int max_blocks) {
  gdn2::CacheView c;
  c.k = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  c.v = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  c.k_scale = const_cast<float*>(k_scale);
  c.v_scale = const_cast<float*>(v_scale);
  c.block_table = block_table;
  c.seq_lens = seq_lens;
  c.cu_seqlens = cu_seqlens;
  c.N = N;
  c.T = T;
  c.P = P;
  c.max_blocks = max_blocks;
  return c;
}

int norm_rope(const void* q, const void* k, const void* gq, const void* gk, const float* q_weight,
              const float* k_weight, const int32_t* positions, const float* inv_freq, void* q_out,
              void* k_out, float* dq_weight, float* dk_weight, int B, int T, int Hq, int Hk, int d,
              long q_stride, long k_stride, int rot, float eps, int flags, int dtype,
              void* workspace, size_t workspace_bytes, void* stream, bool backward) {
  const int st = check_rows(Hq, Hk, d, rot, eps, flags, dtype, inv_freq, q_weight, k_weight);
  if (st != GDN2_OK) return st;
  if (B < 0 || T < 0 || (long)B * T > (long)INT_MAX) return GDN2_INVALID_ARGUMENT;
  if (!stride_ok(q_stride, Hq, d) || !stride_ok(k_stride, Hk, d)) return GDN2_INVALID_ARGUMENT;
  const long tokens = (long)B * T;
  const bool grads = backward && (dq_weight != nullptr || dk_weight != nullptr);
  if (tokens > 0) {
    if (!q || !k || !q_out || !k_out || (backward && (!gq || !gk))) return GDN2_INVALID_ARGUMENT;
    const void* ptrs[7] = {q, k, gq, gk, q_out, k_out, workspace};
    for (const void* p : ptrs)
      if (!aligned(p, 16)) return GDN2_INVALID_ARGUMENT;
    if (!aligned(positions, 4) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
      return GDN2_INVALID_ARGUMENT;
    if (grads && (workspace == nullptr ||
                  workspace_bytes < gdn2::norm_rope_bwd_partial_bytes(tokens, Hq, Hk, d)))
      return GDN2_WORKSPACE_TOO_SMALL;
  }
  if (tokens == 0) return GDN2_OK;
  gdn2::NormRopeArgs a;
  a.q = q; a.k = k; a.gq = gq; a.gk = gk;
  a.q_weight = q_weight; a.k_weight = k_weight;
  a.positions = positions; a.inv_freq = inv_freq;
  a.q_out = q_out; a.k_out = k_out;
  a.dq_weight = dq_weight; a.dk_weight = dk_weight;
  a.partial = grads ? static_cast<float*>(workspace) : nullptr;
  a.tokens = tokens; a.q_stride = q_stride; a.k_stride = k_stride;
  a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot; a.eps = eps;
  a.norm = (flags & GDN2_ROPE_NO_NORM) == 0;
  a.interleaved = (flags & GDN2_ROPE_INTERLEAVED) != 0;
  a.dtype = dtype; a.stream = stream;
  return status_of(backward ? gdn2::launch_norm_rope_bwd(a) : gdn2::launch_norm_rope(a));
}

}  // namespace

extern "C" {

int gdn2_qk_norm_rope(const void* q, const void* k, const float* q_weight, const float* k_weight,
                      const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                      int B, int T, int Hq, int Hk, int d, int64_t q_stride, int64_t k_stride,
                      int rot, float eps, int flags, int dtype, void* hip_stream) {
  return norm_rope(q, k, nullptr, nullptr, q_weight, k_weight, positions, inv_freq, q_out, k_out,
                   nullptr, nullptr, B, T, Hq, Hk, d, q_stride, k_stride, rot, eps, flags, dtype,
                   nullptr, 0, hip_stream, false);
}

int gdn2_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                          const float* q_weight, const float* k_weight, const int32_t* positions,
                          const float* inv_freq, void* dq, void* dk, float* dq_weight,
                          float* dk_weight, int B, int T, int Hq, int Hk, int d, int64_t q_stride,
                          int64_t k_stride, int rot, float eps, int flags, int dtype,
                          void* workspace, size_t workspace_bytes, void* hip_stream) {
  return norm_rope(q, k, dq_out, dk_out, q_weight, k_weight, positions, inv_freq, dq, dk,
                   dq_weight, dk_weight, B, T, Hq, Hk, d, q_stride, k_stride, rot, eps, flags,
                   dtype, workspace, workspace_bytes, hip_stream, true);
}

size_t gdn2_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d) {
  if (B < 0 || T < 0 || Hq <= 0 || Hk <= 0 || !width_ok(d) || (long)B * T > (long)INT_MAX) return 0;
  return gdn2::norm_rope_bwd_partial_bytes((long)B * T, Hq, Hk, d);
}

int gdn2_attn_prologue(const void* q, const void* k, const void* v, const float* q_weight,
                       const float* k_weight, const float* inv_freq, void* q_out, void* k_cache,
                       void* v_cache, float* k_scale, float* v_scale, const int32_t* block_table,
                       const int32_t* seq_lens, const int32_t* cu_seqlens, int B, int T, int Hq,
                       int Hk, int d, int N, int P, int max_blocks, int64_t q_stride,
                       int64_t k_stride, int64_t v_stride, int rot, float eps, int flags,
                       int dtype, void* hip_stream) {
  int st = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, B, T,
                       Hq, Hk, d, N, P, max_blocks, dtype);
  if (st != GDN2_OK) return st;
  st = check_rows(Hq, Hk, d, rot, eps, flags, dtype, inv_freq, q_weight, k_weight);
  if (st != GDN2_OK) return st;
  if (!stride_ok(q_stride, Hq, d) || !stride_ok(k_stride, Hk, d) || !stride_ok(v_stride, Hk, d))
    return GDN2_INVALID_ARGUMENT;
  if (N == 0 || T == 0) return GDN2_OK;
  if (!q || !k || !v || !q_out) return GDN2_INVALID_ARGUMENT;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return GDN2_INVALID_ARGUMENT;
  gdn2::AttnPrologueArgs a;
  a.q = q; a.k = k; a.v = v;
  a.q_weight = q_weight; a.k_weight = k_weight; a.inv_freq = inv_freq; a.q_out = q_out;
  a.c = view(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, T, N, P,
             max_blocks);
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot; a.eps = eps;
  a.norm = (flags & GDN2_ROPE_NO_NORM) == 0;
  a.interleaved = (flags & GDN2_ROPE_INTERLEAVED) != 0;
  a.stream = hip_stream;
  if (gdn2::attn_prologue_groups(a) > (long)INT_MAX) return GDN2_INVALID_ARGUMENT;
  return status_of(gdn2::launch_attn_prologue(a));
}

int gdn2_cache_attention(const void* q, const void* k_cache, const void* v_cache,
                         const float* k_scale, const float* v_scale, const int32_t* block_table,
                         const int32_t* seq_lens, const int32_t* cu_seqlens, void* o, int B, int T,
                         int Hq, int Hk, int d, int N, int P, int max_blocks, int window,
                         float scale, int dtype, void* workspace, size_t workspace_bytes,
                         void* hip_stream) {
  const int st = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens,
                             B, T, Hq, Hk, d, N, P, max_blocks, dtype);
  if (st != GDN2_OK) return st;
  if (window < 0 || !std::isfinite(scale) || !(scale > 0.f)) return GDN2_INVALID_ARGUMENT;
  if (N == 0 || T == 0) return GDN2_OK;
  if (!q || !o || !aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 16))
    return GDN2_INVALID_ARGUMENT;
  const long tokens = (long)B * T;
  if (tokens * Hq > (long)INT_MAX - 1024) return GDN2_INVALID_ARGUMENT;  // rows, in whole tiles
  const gdn2::CacheAttnPlan p =
      gdn2::cache_attn_plan(cu_seqlens != nullptr, N, T, Hq, Hk, d, max_blocks, window);
  if (gdn2::cache_attn_groups(p, cu_seqlens != nullptr, N, Hk) > (long)INT_MAX)
    return GDN2_INVALID_ARGUMENT;
  const size_t need = gdn2::cache_attn_workspace_bytes(p, tokens, Hq, d);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return GDN2_WORKSPACE_TOO_SMALL;
  gdn2::CacheAttnArgs a;
  a.q = q; a.o = o;
  a.c = view(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, T, N, P,
             max_blocks);
  a.Hq = Hq; a.Hk = Hk; a.d = d; a.window = window; a.scale = scale;
  a.workspace = workspace; a.stream = hip_stream;
  return status_of(gdn2::launch_cache_attn(a, p));
}

size_t gdn2_cache_attention_workspace_bytes(int packed, int B, int T, int Hq, int Hk, int d, int N,
                                            int max_blocks, int window) {
  if (B < 0 || T < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk != 0 || !width_ok(d) || N <= 0 ||
      max_blocks <= 0 || window < 0 || (packed ? B != 1 : N != B) || T == 0 ||
      (long)B * T > (long)INT_MAX)
    return 0;
  return gdn2::cache_attn_workspace_bytes(
      gdn2::cache_attn_plan(packed != 0, N, T, Hq, Hk, d, max_blocks, window), (long)B * T, Hq, d);
}

}  // extern "C"
