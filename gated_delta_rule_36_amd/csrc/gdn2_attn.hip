// Softmax attention over the paged 8-bit cache on gfx950.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j  over the keys j in (p_i - window, p_i],
// p_i the position of query i; Hq / Hk query heads share a kv head. Keys and values are e4m3
// with one power of two per (64-token block, head); v_cvt_scalef32_pk_bf16_fp8 turns a pair of
// codes and that power into two bf16 without rounding, so everything after the conversion is
// bf16 attention on exact operands: bf16 MFMA, fp32 scores, running maximum, sum and output.
//
// Both kernels compute the transposed tiles S^T = K Q^T and O^T = V^T P^T: a lane then holds
// scores of one query only, its maximum and scale factor are its own registers, and its scores
// are, in the order the MFMA left them, the B operand of the second product once V^T presents
// its keys in the same order (the cache stores value columns so). No transpose and no exchange
// beyond the row maximum.
//
//  * few rows (a decoded token, a few drafts): all query rows of a (sequence, kv head) fit one
//    or two 16-column tiles; bound by reading the cache. Each wave owns whole blocks, straight
//    from global memory to registers, with no barrier until the waves merge; the key axis is
//    cut over workgroups.
//  * many rows (prompts): 128 query rows a workgroup, 32 a wave, blocks converted once to bf16
//    in LDS (double buffered); bound by the matrix cores and exp2.
// Where the key axis is cut, each piece leaves (maximum, sum, output) in the workspace and a
// merge kernel joins them in a fixed order.

#include "gdn2_attn_device.h"

namespace gdn2 {

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

// 8 codes -> 8 bf16, times the power of two s (exact).
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t lo, uint32_t hi, float s) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Block b of sequence n: its slot, or -1 where the table names none.
__device__ __forceinline__ int block_slot(const CacheView& C, const int* table, int b) {
  const int s = table[b];
  return (unsigned)s < (unsigned)C.P ? s : -1;
}

// Lowest key position that a query at position p sees, minus one.
__device__ __forceinline__ int below_window(int p, int window) {
  return window > 0 && p >= window ? p - window : -1;
}

struct Pieces {
  float* o;   // [splits][rows][D]
  float* ml;  // [splits][rows][2]
  long rows;  // tokens * Hq
  int splits;
};

// ---------------------------------------------------------------- few rows

// grid N * Hk * splits; 4 waves, wave w takes blocks w, w + 4, ... of the piece. RT tiles of 16
// query rows; row r is query token r / G, head h G + r % G. LDS only for the merge of the waves.
template <int D, int RT>
__global__ void __launch_bounds__(256)
gdn2_cache_attn_rows_kernel(CacheAttnArgs A, int split_blocks, Pieces W) {
  constexpr int KH = D / 64;   // 64-channel halves of a key row
  constexpr int DT = D / 16;   // value tiles
  const CacheView& C = A.c;
  const int lane = threadIdx.x & 63, col = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int piece = blockIdx.x % W.splits;
  const int nh = blockIdx.x / W.splits;
  const int h = nh % A.Hk, n = nh / A.Hk;
  const int G = A.Hq / A.Hk;
  const SeqSpan s = seq_span(C, n);
  const int rows = s.count * G < RT * 16 ? s.count * G : RT * 16;
  if (rows == 0) return;
  const int p0 = s.len - s.count;  // position of the first query
  const long span = (long)C.max_blocks * kCacheBlock;
  const int hi = s.len < span ? s.len : (int)span;
  const int lo = below_window(p0, A.window) + 1;
  const int b0 = lo / kCacheBlock + piece * split_blocks;
  int b1 = (hi + kCacheBlock - 1) / kCacheBlock;
  if (b1 > b0 + split_blocks) b1 = b0 + split_blocks;

  auto row_index = [&](int r) {  // row of the [tokens * Hq] output
    return ((long)s.first + r / G) * A.Hq + h * G + r % G;
  };
  if (b0 >= b1) {  // nothing here: an empty piece (the only one: zeros)
    for (int r = threadIdx.x / 16; r < rows; r += 16) {
      if (W.splits == 1) {
        for (int d = (threadIdx.x % 16) * 8; d < D; d += 128)
          *reinterpret_cast<uint4*>((bf16*)A.o + row_index(r) * D + d) = make_uint4(0, 0, 0, 0);
      } else if (threadIdx.x % 16 == 0) {
        float* ml = W.ml + ((long)piece * W.rows + row_index(r)) * 2;
        ml[0] = kNegInf;
        ml[1] = 0.f;
      }
    }
    return;
  }

  // Q^T as the B operand: column r, channels in the order a lane reads a key row (16 bytes of
  // each 64-channel half).
  bf16x8 qf[RT][KH][2];
  int pos[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = t * 16 + col;
    pos[t] = r < rows ? p0 + r / G : -1;
    const bf16* qr = (const bf16*)A.q + row_index(r < rows ? r : 0) * D;
#pragma unroll
    for (int k = 0; k < KH; ++k)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        qf[t][k][u] = *reinterpret_cast<const bf16x8*>(qr + k * 64 + c * 16 + u * 8);
  }

  const int* table = C.block_table + (long)n * C.max_blocks;
  const float scale = A.scale * kLog2e;
  f4 o[RT][DT];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) o[t][i] = f4{0.f, 0.f, 0.f, 0.f};
  }

  uint4 kr[4][KH], vr[DT];
  float ks = 1.f, vs = 1.f;
  auto load_k = [&](int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint8_t* p = C.k + head * (kCacheBlock * D) + col * D + c * 16;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < KH; ++k)
        kr[t][k] = *reinterpret_cast<const uint4*>(p + t * 16 * D + k * 64);
    ks = C.k_scale[head];
  };
  auto load_v = [&](int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint8_t* p = C.v + head * (kCacheBlock * D) + col * kCacheBlock + c * 16;
#pragma unroll
    for (int i = 0; i < DT; ++i)
      vr[i] = *reinterpret_cast<const uint4*>(p + i * 16 * kCacheBlock);
    vs = C.v_scale[head];
  };

  int b = b0 + wave;
  int slot = -1, next = -1;
  if (b < b1) {
    slot = block_slot(C, table, b);
    load_k(slot);
    load_v(slot);
    if (b + 4 < b1) next = block_slot(C, table, b + 4);
  }
  for (; b < b1; b += 4) {
    int after = -1;
    if (b + 8 < b1) after = block_slot(C, table, b + 8);
    f4 sc[RT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int q = 0; q < RT; ++q) sc[q][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const bf16x8 k0 = codes_to_bf16(kr[t][k].x, kr[t][k].y, ks);
        const bf16x8 k1 = codes_to_bf16(kr[t][k].z, kr[t][k].w, ks);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          sc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[q][k][0], sc[q][t], 0, 0, 0);
          sc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[q][k][1], sc[q][t], 0, 0, 0);
        }
      }
    }
    if (b + 4 < b1) load_k(next);

    const int key0 = b * kCacheBlock;
    if (slot < 0 || key0 + kCacheBlock - 1 > p0 ||
        key0 <= below_window(s.len - 1, A.window)) {
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        const int low = below_window(pos[q], A.window);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + t * 16 + c * 4 + i;
            if (slot < 0 || key > pos[q] || key <= low) sc[q][t][i] = kNegInf;
          }
      }
    }
    bf16x8 ph[RT][2], pl[RT][2];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      float top = kNegInf;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[q][t][i]);
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float mn = fmaxf(m[q], top * scale);
      const float base = mn == kNegInf ? 0.f : mn;
      const float alpha = exp2_f(m[q] - base);
      m[q] = mn;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // The weight goes to the matrix cores as two bf16, so that its rounding does not
          // show beside the output's own (the kernel waits on memory, not on MFMA).
          const float p = exp2_f(fmaf(sc[q][t][i], scale, -base));
          sum += p;
          const bf16 hi_p = static_cast<bf16>(p);
          ph[q][t >> 1][(t & 1) * 4 + i] = hi_p;
          pl[q][t >> 1][(t & 1) * 4 + i] = static_cast<bf16>(p - static_cast<float>(hi_p));
        }
      l[q] = l[q] * alpha + sum;
      if (__any(alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < DT; ++i) o[q][i] *= alpha;
      }
    }
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const bf16x8 v0 = codes_to_bf16(vr[i].x, vr[i].y, vs);
      const bf16x8 v1 = codes_to_bf16(vr[i].z, vr[i].w, vs);
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, ph[q][0], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, ph[q][1], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[q][0], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[q][1], o[q][i], 0, 0, 0);
      }
    }
    if (b + 4 < b1) load_v(next);
    slot = next;
    next = after;
  }

  // Merge of the four waves, a tile of rows at a time.
  __shared__ float sm[4][RT * 16], sl[4][RT * 16];
  __shared__ __align__(16) float so[4][16][D + 4];
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    l[q] += __shfl_xor(l[q], 16, 64);
    l[q] += __shfl_xor(l[q], 32, 64);
    if (c == 0) {
      sm[wave][q * 16 + col] = m[q];
      sl[wave][q * 16 + col] = l[q];
    }
  }
  const int tr = threadIdx.x >> 4, ts = threadIdx.x & 15;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    __syncthreads();
    const int rc = q * 16 + col;
    const float top = fmaxf(fmaxf(sm[0][rc], sm[1][rc]), fmaxf(sm[2][rc], sm[3][rc]));
    const float f = m[q] == kNegInf ? 0.f : exp2_f(m[q] - top);
#pragma unroll
    for (int i = 0; i < DT; ++i)
      *reinterpret_cast<f4*>(&so[wave][col][i * 16 + c * 4]) = o[q][i] * f;
    __syncthreads();
    const int r = q * 16 + tr;
    if (r >= rows) continue;
    const float mt = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
    float lt = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      lt += sl[w][r] * (sm[w][r] == kNegInf ? 0.f : exp2_f(sm[w][r] - mt));
    const long out = row_index(r);
    constexpr int E = D / 16;  // channels a thread
    float x[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
      x[i] = (so[0][tr][ts * E + i] + so[1][tr][ts * E + i]) +
             (so[2][tr][ts * E + i] + so[3][tr][ts * E + i]);
    if (W.splits == 1) {
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      bf16* dst = (bf16*)A.o + out * D + ts * E;
#pragma unroll
      for (int i = 0; i < E; i += 4)
        *reinterpret_cast<bf16x4*>(dst + i) =
            bf16x4{static_cast<bf16>(x[i] * inv), static_cast<bf16>(x[i + 1] * inv),
                   static_cast<bf16>(x[i + 2] * inv), static_cast<bf16>(x[i + 3] * inv)};
    } else {
      float* dst = W.o + ((long)piece * W.rows + out) * D + ts * E;
#pragma unroll
      for (int i = 0; i < E; i += 4)
        *reinterpret_cast<f4*>(dst + i) = f4{x[i], x[i + 1], x[i + 2], x[i + 3]};
      if (ts == 0) {
        float* ml = W.ml + ((long)piece * W.rows + out) * 2;
        ml[0] = mt;
        ml[1] = lt;
      }
    }
  }
}

// ---------------------------------------------------------------- many rows

constexpr int kTileRows = 128;

// grid splits * units * Hk; a unit is one 128-row tile of a sequence, the last tiles (with the
// most keys) first. Wave w owns rows 32 w ..; lane: query row (lane % 32), half hf = lane / 32.
template <int D>
__global__ void __launch_bounds__(256, 2)
gdn2_cache_attn_tile_kernel(CacheAttnArgs A, int units, int tiles_per_seq, Pieces W) {
  constexpr int QS = D / 16;       // K steps of the score product
  constexpr int DT = D / 32;       // value tiles
  constexpr int KLD = D + 8;       // LDS rows padded by 16 bytes: reads of 8 rows a phase hit
  constexpr int VLD = kCacheBlock + 8;  // every bank once
  constexpr int NC = kCacheBlock * D / 16 / 256;  // 16-byte chunks a thread stages
  __shared__ __align__(16) bf16 lk[2][kCacheBlock * KLD];
  __shared__ __align__(16) bf16 lv[2][D * VLD];
  const CacheView& C = A.c;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = A.Hq / A.Hk;
  const int h = blockIdx.x % A.Hk;
  const int piece = blockIdx.x / A.Hk / units;
  const int unit = units - 1 - blockIdx.x / A.Hk % units;
  int n, tile;
  if (C.cu_seqlens == nullptr) {
    n = unit % C.N;
    tile = unit / C.N;
  } else {
    n = wave_search(C.N, unit, [&](int i) {
      return (long)clamped_offset(C.cu_seqlens, i, C.T) * G / kTileRows + i;
    });
    tile = unit - (int)((long)clamped_offset(C.cu_seqlens, n, C.T) * G / kTileRows) - n;
  }
  const SeqSpan s = seq_span(C, n);
  const long rows = (long)s.count * G;
  const long row0 = (long)tile * kTileRows;
  if (tile < 0 || row0 >= rows) return;
  const long row_end = row0 + kTileRows < rows ? row0 + kTileRows : rows;
  const int p0 = s.len - s.count;  // position of the first query of the sequence
  const int pmin = p0 + (int)(row0 / G), pmax = p0 + (int)((row_end - 1) / G);
  const long span = (long)C.max_blocks * kCacheBlock;
  const int hi = pmax + 1 < span ? pmax + 1 : (int)span;
  int b0 = (below_window(pmin, A.window) + 1) / kCacheBlock;
  int b1 = hi > 0 ? (hi + kCacheBlock - 1) / kCacheBlock : 0;
  if (W.splits > 1 && b1 > b0) {
    const int per = (b1 - b0 + W.splits - 1) / W.splits;
    b0 += piece * per;
    b1 = b1 < b0 + per ? b1 : b0 + per;
  }

  const long r = row0 + wave * 32 + col;
  const bool live = r < rows;
  const int pos = live ? p0 + (int)(r / G) : -1;
  const long out = ((long)s.first + (live ? r / G : 0)) * A.Hq + h * G + (live ? r % G : 0);
  // positions that this wave's rows span (uniform)
  const long wr0 = row0 + wave * 32;
  const int wmin = wr0 < rows ? p0 + (int)(wr0 / G) : -1;
  const int wmax = wr0 < rows ? p0 + (int)(((wr0 + 31 < rows ? wr0 + 31 : rows - 1)) / G) : -1;
  const int low = below_window(pos, A.window);

  bf16x8 qf[QS];
  {
    const bf16* qr = (const bf16*)A.q + out * D + hf * 8;
#pragma unroll
    for (int u = 0; u < QS; ++u) qf[u] = *reinterpret_cast<const bf16x8*>(qr + u * 16);
  }
  const float scale = A.scale * kLog2e;
  f16v o[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
  float m = kNegInf, l = 0.f;

  const int* table = C.block_table + (long)n * C.max_blocks;
  uint4 kreg[NC], vreg[NC];
  float ks = 1.f, vs = 1.f;
  auto fetch = [&](int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint4* pk = reinterpret_cast<const uint4*>(C.k + head * (kCacheBlock * D));
    const uint4* pv = reinterpret_cast<const uint4*>(C.v + head * (kCacheBlock * D));
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      kreg[j] = pk[tid + j * 256];
      vreg[j] = pv[tid + j * 256];
    }
    ks = C.k_scale[head];
    vs = C.v_scale[head];
  };
  // Chunks to LDS as bf16. Value chunk cc holds the 4-token groups (t, cc), keys 16 t + 4 cc ..:
  // they go where the lane of half cc & 1 reads step t of the second product.
  auto put = [&](int buf) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int i = tid + j * 256;
      bf16* dk = &lk[buf][(i / (D / 16)) * KLD + (i % (D / 16)) * 16];
      *reinterpret_cast<bf16x8*>(dk) = codes_to_bf16(kreg[j].x, kreg[j].y, ks);
      *reinterpret_cast<bf16x8*>(dk + 8) = codes_to_bf16(kreg[j].z, kreg[j].w, ks);
      const int cc = i & 3;
      bf16* dv = &lv[buf][(i >> 2) * VLD + (cc & 1) * 8 + (cc >> 1) * 4];
      const bf16x8 a = codes_to_bf16(vreg[j].x, vreg[j].y, vs);
      const bf16x8 b = codes_to_bf16(vreg[j].z, vreg[j].w, vs);
      *reinterpret_cast<bf16x4*>(dv) = __builtin_shufflevector(a, a, 0, 1, 2, 3);
      *reinterpret_cast<bf16x4*>(dv + 16) = __builtin_shufflevector(a, a, 4, 5, 6, 7);
      *reinterpret_cast<bf16x4*>(dv + 32) = __builtin_shufflevector(b, b, 0, 1, 2, 3);
      *reinterpret_cast<bf16x4*>(dv + 48) = __builtin_shufflevector(b, b, 4, 5, 6, 7);
    }
  };

  int slot = -1, next = -1;
  if (b0 < b1) {
    slot = block_slot(C, table, b0);
    fetch(slot);
    if (b0 + 1 < b1) next = block_slot(C, table, b0 + 1);
    put(0);
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    const int buf = (b - b0) & 1;
    const bool more = b + 1 < b1;
    int after = -1;
    if (more) fetch(next);
    if (b + 2 < b1) after = block_slot(C, table, b + 2);
    const int key0 = b * kCacheBlock;
    // rows of this wave that see something of the block
    if (slot >= 0 && key0 <= wmax && key0 + kCacheBlock - 1 > below_window(wmin, A.window)) {
      f16v sc[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int j = 0; j < 16; ++j) sc[t][j] = 0.f;
#pragma unroll
        for (int u = 0; u < QS; ++u) {
          const bf16x8 kf = *reinterpret_cast<const bf16x8*>(
              &lk[buf][(t * 32 + col) * KLD + u * 16 + hf * 8]);
          sc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[u], sc[t], 0, 0, 0);
        }
      }
      if (key0 + kCacheBlock - 1 > wmin || key0 <= below_window(wmax, A.window)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int key = key0 + t * 32 + (j >> 2) * 8 + hf * 4 + (j & 3);
            if (key > pos || key <= low) sc[t][j] = kNegInf;
          }
      }
      float top = kNegInf;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, sc[t][j]);
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float mn = fmaxf(m, top * scale);
      const float base = mn == kNegInf ? 0.f : mn;
      const float alpha = exp2_f(m - base);
      m = mn;
      float sum = 0.f;
      bf16x8 pf[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          // one rounding of the weight to bf16 (at most 2^-8 of it), the matrix cores' input type
          const float p = exp2_f(fmaf(sc[t][j], scale, -base));
          sum += p;
          pf[t * 2 + (j >> 3)][j & 7] = static_cast<bf16>(p);
        }
      l = l * alpha + sum;
      if (__any(alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] *= alpha;
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf16x8 vf = *reinterpret_cast<const bf16x8*>(
              &lv[buf][(i * 32 + col) * VLD + u * 16 + hf * 8]);
          o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf, pf[u], o[i], 0, 0, 0);
        }
    }
    if (more) put(buf ^ 1);
    slot = next;
    next = after;
    __syncthreads();
  }

  l += __shfl_xor(l, 32, 64);
  if (!live) return;
  if (W.splits == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    bf16* dst = (bf16*)A.o + out * D + hf * 4;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<bf16x4*>(dst + i * 32 + j * 8) =
            bf16x4{static_cast<bf16>(o[i][j * 4] * inv), static_cast<bf16>(o[i][j * 4 + 1] * inv),
                   static_cast<bf16>(o[i][j * 4 + 2] * inv),
                   static_cast<bf16>(o[i][j * 4 + 3] * inv)};
  } else {
    if (hf == 0) {
      float* ml = W.ml + ((long)piece * W.rows + out) * 2;
      ml[0] = m;
      ml[1] = l;
    }
    float* dst = W.o + ((long)piece * W.rows + out) * D + hf * 4;
    if (l != 0.f) {
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f4*>(dst + i * 32 + j * 8) =
              f4{o[i][j * 4], o[i][j * 4 + 1], o[i][j * 4 + 2], o[i][j * 4 + 3]};
    }
  }
}

// ---------------------------------------------------------------- merge of the pieces

// D / 4 lanes a row, pieces in order; a piece without keys (sum 0) left no output.
template <int D>
__global__ void __launch_bounds__(256) gdn2_cache_attn_merge_kernel(CacheAttnArgs A, Pieces W) {
  constexpr int LN = D / 4;
  const long row = (long)blockIdx.x * (256 / LN) + threadIdx.x / LN;
  const int l = threadIdx.x % LN;
  if (row >= W.rows) return;
  if (A.c.cu_seqlens != nullptr) {  // rows outside the sequences are left as they are
    const long tok = row / A.Hq;
    if (tok < clamped_offset(A.c.cu_seqlens, 0, A.c.T) ||
        tok >= clamped_offset(A.c.cu_seqlens, A.c.N, A.c.T))
      return;
  }
  float top = kNegInf;
  for (int p = l; p < W.splits; p += LN) {
    const float* ml = W.ml + ((long)p * W.rows + row) * 2;
    if (ml[1] != 0.f) top = fmaxf(top, ml[0]);
  }
#pragma unroll
  for (int k = 1; k < LN; k <<= 1) top = fmaxf(top, __shfl_xor(top, k, 64));
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int p = 0; p < W.splits; ++p) {
    const float* ml = W.ml + ((long)p * W.rows + row) * 2;
    const float lp = ml[1];
    if (lp == 0.f) continue;
    const float f = exp2_f(ml[0] - top);
    sum += lp * f;
    acc += *reinterpret_cast<const f4*>(W.o + ((long)p * W.rows + row) * D + l * 4) * f;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<bf16x4*>((bf16*)A.o + row * D + l * 4) =
      bf16x4{static_cast<bf16>(acc[0] * inv), static_cast<bf16>(acc[1] * inv),
             static_cast<bf16>(acc[2] * inv), static_cast<bf16>(acc[3] * inv)};
}

template <int D>
hipError_t run(const CacheAttnArgs& a, const CacheAttnPlan& p) {
  const hipStream_t st = (hipStream_t)a.stream;
  const long tokens = a.c.cu_seqlens ? a.c.T : (long)a.c.N * a.c.T;
  Pieces w;
  w.rows = tokens * a.Hq;
  w.splits = p.splits;
  w.o = (float*)a.workspace;
  w.ml = w.o + (size_t)p.splits * w.rows * D;
  if (p.few_rows) {
    const dim3 grid((unsigned)((long)a.c.N * a.Hk * p.splits));
    if (p.row_tiles == 1)
      hipLaunchKernelGGL((gdn2_cache_attn_rows_kernel<D, 1>), grid, dim3(256), 0, st, a,
                         p.split_blocks, w);
    else
      hipLaunchKernelGGL((gdn2_cache_attn_rows_kernel<D, 2>), grid, dim3(256), 0, st, a,
                         p.split_blocks, w);
  } else {
    const int units = a.c.cu_seqlens ? p.row_tiles : p.row_tiles * a.c.N;
    hipLaunchKernelGGL((gdn2_cache_attn_tile_kernel<D>),
                       dim3((unsigned)((long)units * a.Hk * p.splits)), dim3(256), 0, st, a,
                       units, p.row_tiles, w);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  constexpr int RPB = 256 / (D / 4);
  hipLaunchKernelGGL((gdn2_cache_attn_merge_kernel<D>), dim3((unsigned)((w.rows + RPB - 1) / RPB)),
                     dim3(256), 0, st, a, w);
  return hipGetLastError();
}

}  // namespace

CacheAttnPlan cache_attn_plan(bool packed, int N, int T, int Hq, int Hk, int d, int max_blocks,
                              int window) {
  CacheAttnPlan p;
  const long G = Hq / Hk, rows = T * G;
  // blocks that one call can reach: the table's, or what the window and the new tokens span
  long nb = max_blocks;
  if (window > 0) {
    const long w = ((long)window + T + kCacheBlock - 3) / kCacheBlock + 1;
    if (w < nb) nb = w;
  }
  // The lengths are on the device, so the cut goes by the table's width; pieces past a
  // sequence's end leave at once.
  p.few_rows = rows <= 32;
  if (p.few_rows) {
    p.row_tiles = rows <= 16 ? 1 : 2;
    long per = nb * N * Hk / 2048;  // about 8 workgroups a compute unit
    if (per < nb / 256) per = nb / 256;
    per = (per + 3) / 4 * 4;  // a block a wave
    if (per < 4) per = 4;
    p.split_blocks = (int)per;
    p.splits = (int)((nb + per - 1) / per);
  } else {
    p.row_tiles = packed ? (int)(rows / kTileRows + N) : (int)((rows + kTileRows - 1) / kTileRows);
    p.split_blocks = 0;
    const long wgs = (packed ? p.row_tiles : (long)p.row_tiles * N) * Hk;
    long s = 512 / wgs;  // two workgroups a compute unit
    if (s > (nb + 3) / 4) s = (nb + 3) / 4;
    p.splits = s < 1 ? 1 : (int)s;
  }
  if (p.splits < 1) p.splits = 1;
  return p;
}

size_t cache_attn_workspace_bytes(const CacheAttnPlan& p, long tokens, int Hq, int d) {
  if (p.splits == 1) return 0;
  return (size_t)p.splits * tokens * Hq * (d + 2) * sizeof(float);
}

long cache_attn_groups(const CacheAttnPlan& p, bool packed, int N, int Hk) {
  const long units = p.few_rows ? N : packed ? p.row_tiles : (long)p.row_tiles * N;
  return units * Hk * p.splits;
}

hipError_t launch_cache_attn(const CacheAttnArgs& a, const CacheAttnPlan& p) {
  return a.d == 64 ? run<64>(a, p) : run<128>(a, p);
}

}  // namespace gdn2
