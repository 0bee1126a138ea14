// Host-side argument blocks and launchers of what stands around the mixer in a stack: the diagonal
// gated recurrence, the norm between layers with the residual's addition, and the verification of
// drafted tokens.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn2 {

constexpr long kMaxGroups = (1L << 23) - 1;  // of a launch: 512 threads each stay below 2^32

// ---- diagonal recurrence: h = exp(g) h + w v, a state per channel

// How sequences are cut: into units of seg tokens.
struct RecurrenceCut {
  bool cut;          // some sequence may have more than one unit
  int seg;           // tokens of a unit
  int per_sequence;  // units of a sequence (packed batches: see the kernels)
  int units;
  bool twice;        // forward: two passes of the outputs, none for the maps alone
  float* maps;       // workspace, where cut: [units, 2, D], then int [units, strips] (for `twice`)
};
struct RecurrenceArgs {
  const void *v, *g, *w;      // [tokens, D], rows dense, one stride each; w may be null (ones)
  const float* s0;            // [N, D] or null
  void* o;                    // [tokens, D] dense, or null
  float* sN;                  // [N, D] or null
  float* states;              // [slots, D]: the state before every kStateTokens tokens, or null
  const int32_t* cu_seqlens;  // [N + 1] or null
  long v_stride, g_stride, w_stride;
  int T, N, D, dtype;         // T: tokens of a sequence, or in all when packed
  RecurrenceCut cut;
  bool zero_rest;             // set by the launchers: zeros to the rows of no sequence,
  bool shared_lines;          // rows that do not begin at lines of 128 bytes
  void* stream;
};
struct RecurrenceBwdArgs {
  RecurrenceArgs f;  // v, g, w, states, the sizes
  const void* d_o;   // [tokens, D] dense
  const float* d_sN;  // [N, D] or null
  void *dv, *dg, *dw;  // dense
  float* d_s0;        // [N, D] or null
};
struct RecurrenceTokensArgs {
  const void *v, *g, *w;
  float* pool;
  const int32_t *indices, *commit;
  void* o;
  float* step_states;
  long v_stride, g_stride, w_stride;
  int N, L, D, P, dtype;
  void* stream;
};

// Kept states: one before every kStateTokens tokens of a sequence. Sequence n's begin at slot
// n * ceil(T / kStateTokens), packed at cu_seqlens[n] / kStateTokens + n. (Where there are tokens there is
// a slot: the pointer is never null.)
constexpr int kStateTokens = 64;
constexpr int kMaxStride = 1 << 21;  // elements from one token to the next
long recurrence_state_slots(bool packed, int B, int T, int N);
RecurrenceCut recurrence_cut(bool backward, bool packed, int B, int T, int D, int N);
long recurrence_groups(const RecurrenceCut& c, int D);  // workgroups of the largest launch
size_t recurrence_workspace_bytes(const RecurrenceCut& c, int D);
hipError_t launch_recurrence(const RecurrenceArgs& a);
hipError_t launch_recurrence_bwd(const RecurrenceBwdArgs& a);
hipError_t launch_recurrence_tokens(const RecurrenceTokensArgs& a);

// ---- norm between layers: h = x + r, y = h / sqrt(mean(h^2) + eps) * weight
struct ResidualNormArgs {
  const void *x, *r;    // [rows, D], rows dense, one stride each; r may be null (h = x, not written)
  const float* weight;  // [D]
  void *y, *h;          // [rows, D] dense; y: the codes with scale
  float* scale;         // 8-bit output: [rows, D / group], else null
  long rows, x_stride, r_stride;
  int D, group;         // group: channels of a scale (32, 64, 128 or D)
  float eps;
  int dtype, r_dtype;   // of x and y, of r and h
  bool stream_rows;     // set by the launcher: inputs past the caches
  void* stream;
};
struct ResidualNormBwdArgs {
  const void *dy, *dh, *h;  // [rows, D] dense; dh may be null (zero)
  const float* weight;
  void *dx, *dr;            // gradient in x's type and in r's; dr null where the types are the same
  float *dweight, *partial; // [D]; workspace
  long rows, h_stride;
  int D;
  float eps;
  int dtype, r_dtype;
  void* stream;
};
constexpr int kNormMaxWidth = 16384;
int residual_norm_bwd_groups(long rows, int D);  // workgroups, each leaves one partial weight gradient
hipError_t launch_residual_norm(const ResidualNormArgs& a);
hipError_t launch_residual_norm_bwd(const ResidualNormBwdArgs& a);

// ---- verification of drafted tokens
struct VerifyArgs {
  const void *p, *q;  // [N, L + 1, V], [N, L, V] or null (drafts that were certain)
  const int32_t *drafts, *draft_len;  // [N, L], [N] or null (L)
  const float* u;     // [N, L + 1]
  int32_t *tokens, *commit;  // [N, L + 1], [N]
  double* sums;       // workspace [N, pieces, 2]
  int N, L, V, dtype;
  void* stream;
};
int verify_pieces(int V);
hipError_t launch_verify(const VerifyArgs& a);

}  // namespace gdn2
