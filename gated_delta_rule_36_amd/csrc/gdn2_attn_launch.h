// Host-side argument blocks and launchers of the softmax-attention layer: per-head norms with
// the position rotation, the serving prologue that fills the 8-bit cache, and attention over
// that cache.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn2 {

constexpr int kCacheBlock = 64;  // tokens per cache block (one scale per block and head)

struct NormRopeArgs {
  const void *q, *k;                  // [tokens, H, d], rows of a token dense
  const void *gq, *gk;                // backward: gradients of the outputs, dense
  const float *q_weight, *k_weight;   // [d] or null (ones)
  const int32_t* positions;           // [tokens] or null (token index % T)
  const float* inv_freq;              // [rot / 2] (null only when rot = 0)
  void *q_out, *k_out;                // forward: outputs; backward: dq, dk (dense)
  float *dq_weight, *dk_weight;       // backward: [d] or null
  float* partial;                     // backward: workspace
  long tokens, q_stride, k_stride;    // strides: elements from one token to the next
  int T, Hq, Hk, d, rot;
  float eps;
  bool norm, interleaved;
  int dtype;
  void* stream;
};

// Workgroups along the token axis of the backward (each leaves one partial weight gradient).
int norm_rope_bwd_groups(long tokens);
size_t norm_rope_bwd_partial_bytes(long tokens, int Hq, int Hk, int d);
hipError_t launch_norm_rope(const NormRopeArgs& a);
hipError_t launch_norm_rope_bwd(const NormRopeArgs& a);

// The paged cache, as both of its users see it.
struct CacheView {
  uint8_t *k, *v;             // [P, Hk, 64, d], [P, Hk, d, 64 (permuted)] e4m3
  float *k_scale, *v_scale;   // [P, Hk]
  const int32_t* block_table; // [N, max_blocks]
  const int32_t* seq_lens;    // [N], tokens after this call
  const int32_t* cu_seqlens;  // [N + 1] or null
  int N, T, P, max_blocks;    // T: new tokens per sequence, or in all when packed
};

struct AttnPrologueArgs {
  const void *q, *k, *v;
  const float *q_weight, *k_weight, *inv_freq;
  void* q_out;
  CacheView c;
  long q_stride, k_stride, v_stride;
  int Hq, Hk, d, rot;
  float eps;
  bool norm, interleaved;
  void* stream;
};
long attn_prologue_groups(const AttnPrologueArgs& a);  // workgroups of its one launch
hipError_t launch_attn_prologue(const AttnPrologueArgs& a);

struct CacheAttnArgs {
  const void* q;  // [tokens, Hq, d] bf16
  void* o;        // the same
  CacheView c;
  int Hq, Hk, d, window;
  float scale;
  void* workspace;
  void* stream;
};

// How a call is cut: which kernel, and into how many pieces of the key axis.
struct CacheAttnPlan {
  bool few_rows;     // every wave holds all query rows of a (sequence, kv head)
  int row_tiles;     // few_rows: 16-row tiles; else: row tiles (per sequence, or in all)
  int waves;         // few rows: waves of a workgroup
  int tile_rows;     // many rows: query rows of a tile
  int splits;        // pieces of the key axis
  int split_blocks;  // cache blocks per piece
  // Mixed batches: sequences of up to mixed_rows query rows a kv head (16 or 32; 0: no such pass)
  // are left to a second pass of the few-row kernel, with a plan of its own.
  int mixed_rows, mixed_waves, mixed_blocks, mixed_splits;
  long mixed_part_rows;  // rows of its partial results
};
CacheAttnPlan cache_attn_plan(bool packed, int N, int T, int Hq, int Hk, int d, int max_blocks,
                              int window);
size_t cache_attn_workspace_bytes(const CacheAttnPlan& p, long tokens, int Hq, int d);
long cache_attn_groups(const CacheAttnPlan& p, bool packed, int N, int Hk);
hipError_t launch_cache_attn(const CacheAttnArgs& a, const CacheAttnPlan& p);

}  // namespace gdn2
