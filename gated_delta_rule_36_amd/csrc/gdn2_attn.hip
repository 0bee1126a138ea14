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
//  * many rows (prompts): 128 or 256 query rows a workgroup, 32 a wave, blocks converted once to
//    bf16 in LDS (double buffered); bound by the matrix cores and exp2.
// Where the key axis is cut, each piece leaves (maximum, sum, output) in the workspace and a
// merge kernel joins them in a fixed order.

#include "gdn2_attn_device.h"

namespace gdn2 {

namespace {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
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
  const int s = scalar_load(table, b);
  return (unsigned)s < (unsigned)C.P ? s : -1;
}

// 16 bytes of a value block of `bytes` bytes at `base` (wave-uniform), through a buffer whose size is
// zero for a block that does not exist: it reads as zeros, since weights of zero would not keep a NaN
// at `base` out of the product. (Its keys are those at `base`, masked by selection.) That costs
// nothing; a branch around the loads took packed prompts with a window from 44.4 to 47.2 us and single
// tokens with one from 51 to 52.
__device__ __forceinline__ uint4 value_chunk(const uint8_t* base, int bytes, int off) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0, bytes, 0x00020000);
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Lowest key position that a query at position p sees, minus one.
__device__ __forceinline__ int below_window(int p, int window) {
  return window > 0 && p >= window ? p - window : -1;
}

struct Pieces {
  float* o;   // [splits][rows][D]
  float* ml;  // [splits][rows][2]
  long rows;  // tokens * Hq; mixed batches, few rows: few for each (sequence, kv head)
  int splits;
  int few;    // mixed batches: sequences of up to so many query rows a kv head go to the few-row
              // kernel, the others to the many-row one; 0: one kernel has them all
};

// ---------------------------------------------------------------- few rows

// grid N * Hk * splits; NW waves, wave w takes blocks w, w + NW, ... of the piece. RT tiles of 16
// query rows; row r is query token r / G, head h G + r % G. LDS only for the merge of the waves.
template <int D, int RT, int NW>
__global__ void __launch_bounds__(NW * 64, 2)
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
  const int* table = C.block_table + (long)n * C.max_blocks;
  // without a window the first block is known before the length is: one wait for both
  const int e = piece * split_blocks + wave;
  const int early = A.window > 0 ? -1 : block_slot(C, table, e < C.max_blocks ? e : 0);
  const SeqSpan s = seq_span(C, n);
  if (W.few && (long)s.count * G > W.few) return;
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
  auto part_index = [&](int r) { return W.few ? (long)nh * W.few + r : row_index(r); };
  if (b0 >= b1) {  // nothing here: an empty piece (the only one: zeros)
    for (int r = threadIdx.x / 16; r < rows; r += NW * 4) {
      if (W.splits == 1) {
        for (int d = (threadIdx.x % 16) * 8; d < D; d += 128)
          *reinterpret_cast<uint4*>((bf16*)A.o + row_index(r) * D + d) = make_uint4(0, 0, 0, 0);
      } else if (threadIdx.x % 16 == 0) {
        float* ml = W.ml + ((long)piece * W.rows + part_index(r)) * 2;
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

  struct Block {  // a block's codes as a lane holds them
    uint4 k[4][KH], v[DT];
    float ks, vs;
  };
  auto load_k = [&](Block& r, int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint8_t* p = C.k + head * (kCacheBlock * D) + col * D + c * 16;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int k = 0; k < KH; ++k)
        r.k[t][k] = *reinterpret_cast<const uint4*>(p + t * 16 * D + k * 64);
    r.ks = scalar_load(C.k_scale, head);
  };
  auto load_v = [&](Block& r, int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint8_t* p = C.v + head * (kCacheBlock * D);
#pragma unroll
    for (int i = 0; i < DT; ++i)
      r.v[i] = value_chunk(p, slot < 0 ? 0 : kCacheBlock * D, (i * 16 + col) * kCacheBlock + c * 16);
    r.vs = scalar_load(C.v_scale, head);
  };

  // One block's registers, refilled as they are consumed: a second set (the next block's loads
  // before this one's arithmetic) measured 2 to 5% slower.
  int b = b0 + wave;
  int slot = -1, next = -1;
  Block cur;
  if (b < b1) {
    slot = A.window > 0 ? block_slot(C, table, b) : early;
    load_k(cur, slot);
    load_v(cur, slot);
    if (b + NW < b1) next = block_slot(C, table, b + NW);
  }
  for (; b < b1; b += NW) {
    int after = -1;
    if (b + 2 * NW < b1) after = block_slot(C, table, b + 2 * NW);
    f4 sc[RT][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int q = 0; q < RT; ++q) sc[q][t] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const bf16x8 k0 = codes_to_bf16(cur.k[t][k].x, cur.k[t][k].y, cur.ks);
        const bf16x8 k1 = codes_to_bf16(cur.k[t][k].z, cur.k[t][k].w, cur.ks);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          sc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k0, qf[q][k][0], sc[q][t], 0, 0, 0);
          sc[q][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k1, qf[q][k][1], sc[q][t], 0, 0, 0);
        }
      }
    }
    if (b + NW < b1) load_k(cur, next);

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
      top = max_rows(top);
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
    const float vs = slot < 0 ? 1.f : cur.vs;
#pragma unroll
    for (int i = 0; i < DT; ++i) {
      const bf16x8 v0 = codes_to_bf16(cur.v[i].x, cur.v[i].y, vs);
      const bf16x8 v1 = codes_to_bf16(cur.v[i].z, cur.v[i].w, vs);
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, ph[q][0], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, ph[q][1], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[q][0], o[q][i], 0, 0, 0);
        o[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[q][1], o[q][i], 0, 0, 0);
      }
    }
    if (b + NW < b1) load_v(cur, next);
    slot = next;
    next = after;
  }

  // Merge of the waves, a tile of rows at a time.
  __shared__ float sm[NW][RT * 16], sl[NW][RT * 16];
  __shared__ __align__(16) float so[NW][16][D + 4];
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    l[q] += __shfl_xor(l[q], 16, 64);
    l[q] += __shfl_xor(l[q], 32, 64);
    if (c == 0) {
      sm[wave][q * 16 + col] = m[q];
      sl[wave][q * 16 + col] = l[q];
    }
  }
  constexpr int TPR = NW * 4, E = D / TPR;  // threads a row, channels a thread
  const int tr = threadIdx.x / TPR, ts = threadIdx.x % TPR;
#pragma unroll
  for (int q = 0; q < RT; ++q) {
    __syncthreads();
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, sm[w][q * 16 + col]);
    const float f = m[q] == kNegInf ? 0.f : exp2_f(m[q] - top);
#pragma unroll
    for (int i = 0; i < DT; ++i)
      *reinterpret_cast<f4*>(&so[wave][col][i * 16 + c * 4]) = o[q][i] * f;
    __syncthreads();
    const int r = q * 16 + tr;
    if (r >= rows) continue;
    float mt = kNegInf, lt = 0.f, x[E] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) mt = fmaxf(mt, sm[w][r]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      lt += sl[w][r] * (sm[w][r] == kNegInf ? 0.f : exp2_f(sm[w][r] - mt));
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] += so[w][tr][ts * E + i];
    }
    if (W.splits == 1) {
      const float inv = lt == 0.f ? 0.f : 1.f / lt;
      bf16* dst = (bf16*)A.o + row_index(r) * D + ts * E;
#pragma unroll
      for (int i = 0; i < E; ++i) dst[i] = static_cast<bf16>(x[i] * inv);
    } else {
      const long out = part_index(r);
      float* dst = W.o + ((long)piece * W.rows + out) * D + ts * E;
#pragma unroll
      for (int i = 0; i < E; ++i) dst[i] = x[i];
      if (ts == 0) {
        float* ml = W.ml + ((long)piece * W.rows + out) * 2;
        ml[0] = mt;
        ml[1] = lt;
      }
    }
  }
}

// ---------------------------------------------------------------- many rows

// grid splits * units * Hk; a unit is one tile of 32 NW rows of a sequence, the last tiles (with the
// most keys) first. Wave w owns rows 32 w ..; lane: query row (lane % 32), half hf = lane / 32.
//
// The loop is pipelined over two blocks: the softmax of block b (VALU, exp2 above all) runs beside
// the products K(b + 1) Q^T, and the maximum of b + 1 and the staging of K(b + 2) and V(b + 1)
// beside V(b)^T P(b)^T, so that the matrix cores have work throughout.
template <int D, int NW>
__global__ void __launch_bounds__(NW * 64, 2)
gdn2_cache_attn_tile_kernel(CacheAttnArgs A, int units, int split_blocks, Pieces W) {
  constexpr int ROWS = 32 * NW;   // rows of a workgroup
  constexpr int QS = D / 16;       // K steps of the score product
  constexpr int DT = D / 32;       // value tiles
  constexpr int KLD = D + 8;       // LDS rows padded by 16 bytes: reads of 8 rows a phase hit
  constexpr int VLD = kCacheBlock + 8;  // every bank once
  constexpr int NT = NW * 64, NC = kCacheBlock * D / 16 / NT;  // 16-byte chunks a thread stages
  struct Stage {
    bf16 k[2][kCacheBlock * KLD];
    bf16 v[2][D * VLD];
  };
  __shared__ __align__(16) Stage lds;
  static_assert(sizeof(Stage) >= sizeof(bf16) * ROWS * KLD, "room for the rows of the output");
  const CacheView& C = A.c;
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int G = A.Hq / A.Hk;
  const int h = blockIdx.x % A.Hk;
  const int piece = blockIdx.x / A.Hk / units;
  const int unit = units - 1 - blockIdx.x / A.Hk % units;
  int n, tile;
  SeqSpan s;
  if (C.cu_seqlens == nullptr) {
    n = unit % C.N;
    tile = unit / C.N;
    s = seq_span(C, n);
  } else {  // sequence n owns the tiles from floor(first row / ROWS) + n on
    n = packed_span(C, unit, s, [&](int first, int i) { return (long)first * G / ROWS + i; });
    tile = unit - (int)((long)s.first * G / ROWS) - n;
  }
  n = uniform(n);
  tile = uniform(tile);
  s = uniform(s);
  const int rows = s.count * G;  // (at most tokens * Hq, which the host holds below 2^31)
  if (tile < 0 || (long)tile * ROWS >= rows) return;
  if (rows <= W.few) {  // the few-row kernel's (a tile at most): the merge leaves these rows alone
    if (W.splits > 1 && piece == 0 && tid < rows)
      W.ml[(((long)s.first + tid / G) * A.Hq + h * G + tid % G) * 2 + 1] = -1.f;
    return;
  }
  const int row0 = tile * ROWS;
  const int row_last = rows - row0 > ROWS ? row0 + ROWS - 1 : rows - 1;
  const int p0 = s.len - s.count;  // position of the first query of the sequence
  const int pmin = p0 + row0 / G, pmax = p0 + row_last / G;
  const long span = (long)C.max_blocks * kCacheBlock;
  const int hi = pmax + 1 < span ? pmax + 1 : (int)span;
  const int b0 = uniform((below_window(pmin, A.window) + 1) / kCacheBlock + piece * split_blocks);
  int b1 = hi > 0 ? (hi + kCacheBlock - 1) / kCacheBlock : 0;
  b1 = uniform(b1 > b0 + split_blocks ? b0 + split_blocks : b1);

  // positions that this wave's rows span; a wave past the last row has none (-1)
  const int wr0 = row0 + wave * 32;
  const int wr1 = rows - wr0 > 32 ? wr0 + 31 : rows - 1;
  const int wmin = uniform(wr0 < rows ? p0 + wr0 / G : -1);
  const int wmax = uniform(wr0 < rows ? p0 + wr1 / G : -1);
  const int r = wr0 + col;
  const bool live = r < rows;
  const int rt = (live ? r : 0) / G, rh = (live ? r : 0) % G;  // query token, head of the group
  const int pos = live ? p0 + rt : -1;
  const int low = below_window(pos, A.window);
  const long out = ((long)s.first + rt) * A.Hq + h * G + rh;
  bf16x8 qf[QS];
  {
    const bf16* qr = (const bf16*)A.q + out * D + hf * 8;
#pragma unroll
    for (int u = 0; u < QS; ++u) qf[u] = *reinterpret_cast<const bf16x8*>(qr + u * 16);
  }
  const float scale = A.scale * kLog2e;
  f16v o[DT];
  float m = kNegInf, l = 0.f;
#pragma unroll
  for (int i = 0; i < DT; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) o[i][j] = 0.f;

  const int* table = C.block_table + (long)n * C.max_blocks;
  uint4 kreg[NC], vreg[NC];
  float ks = 1.f, vs = 1.f;
  auto fetch_k = [&](int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint4* p = reinterpret_cast<const uint4*>(C.k + head * (kCacheBlock * D));
#pragma unroll
    for (int j = 0; j < NC; ++j) kreg[j] = p[tid + j * NT];
    ks = scalar_load(C.k_scale, head);
  };
  auto fetch_v = [&](int slot) {
    const long head = (long)(slot < 0 ? 0 : slot) * A.Hk + h;
    const uint8_t* p = C.v + head * (kCacheBlock * D);
#pragma unroll
    for (int j = 0; j < NC; ++j)
      vreg[j] = value_chunk(p, slot < 0 ? 0 : kCacheBlock * D, (tid + j * NT) * 16);
    vs = scalar_load(C.v_scale, head);
  };
  auto put_codes = [&](int buf, int j, const uint4& x, float scale_k) {
    const int i = tid + j * NT;
    bf16* dk = &lds.k[buf][(i / (D / 16)) * KLD + (i % (D / 16)) * 16];
    *reinterpret_cast<bf16x8*>(dk) = codes_to_bf16(x.x, x.y, scale_k);
    *reinterpret_cast<bf16x8*>(dk + 8) = codes_to_bf16(x.z, x.w, scale_k);
  };
  auto put_k = [&](int buf, int j) { put_codes(buf, j, kreg[j], ks); };
  // Value chunk cc holds the 4-token groups (t, cc), keys 16 t + 4 cc ..: they go where the lane
  // of half cc & 1 reads step t of the second product.
  auto put_v = [&](int buf, int j, int slot) {
    const int i = tid + j * NT;
    const float s = slot < 0 ? 1.f : vs;
    const int cc = i & 3;
    bf16* dv = &lds.v[buf][(i >> 2) * VLD + (cc & 1) * 8 + (cc >> 1) * 4];
    const bf16x8 a = codes_to_bf16(vreg[j].x, vreg[j].y, s);
    const bf16x8 b = codes_to_bf16(vreg[j].z, vreg[j].w, s);
    *reinterpret_cast<bf16x4*>(dv) = __builtin_shufflevector(a, a, 0, 1, 2, 3);
    *reinterpret_cast<bf16x4*>(dv + 16) = __builtin_shufflevector(a, a, 4, 5, 6, 7);
    *reinterpret_cast<bf16x4*>(dv + 32) = __builtin_shufflevector(b, b, 0, 1, 2, 3);
    *reinterpret_cast<bf16x4*>(dv + 48) = __builtin_shufflevector(b, b, 4, 5, 6, 7);
  };
  // Row of a value tile that a lane reads: bits 2 and 3 exchanged, so that a lane's results
  // j, j + 1 .. j + 7 are 8 neighbouring channels, 16 bytes of the output (j = 0 and 8).
  const int vrow = (col & 0x13) | (col & 4) << 1 | (col & 8) >> 1;
  // Fragment of K step k (u = k / 2: channels 16 u .., t = k % 2: keys 32 t ..) and of V step v
  // (u = v / DT: keys 16 u .., tile v % DT: channels 32 ..).
  auto k_frag = [&](int buf, int k) {
    return *reinterpret_cast<const bf16x8*>(
        &lds.k[buf][((k & 1) * 32 + col) * KLD + (k >> 1) * 16 + hf * 8]);
  };
  auto v_frag = [&](int buf, int v) {
    return *reinterpret_cast<const bf16x8*>(
        &lds.v[buf][((v % DT) * 32 + vrow) * VLD + (v / DT) * 16 + hf * 8]);
  };
  constexpr int STEPS = 2 * QS;  // of either product
  static_assert(STEPS == 4 * DT, "as many K fragments as V fragments");

  if (b0 < b1) {
    f16v sa[2], sb[2];  // scores of one block and of the next, in turn
    // (indices past the last block repeat it: the loads do not wait for a branch)
    const int e = b1 - 1;
    int s0 = block_slot(C, table, b0), s1 = block_slot(C, table, b0 + 1 < b1 ? b0 + 1 : e),
        s2 = block_slot(C, table, b0 + 2 < b1 ? b0 + 2 : e);
    // K(b0), K(b0 + 1) and V(b0) in one wait
    fetch_k(s0);
    const float ks0 = ks;
    uint4 k0[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) k0[j] = kreg[j];
    fetch_k(s1);
    fetch_v(s0);
#pragma unroll
    for (int j = 0; j < NC; ++j) put_codes(0, j, k0[j], ks0);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      put_k(1, j);
      put_v(0, j, s0);
    }
    fetch_k(s2);
    fetch_v(s1);
    __syncthreads();
    const f16v zero = {};
    const bf16 one = static_cast<bf16>(1.f);
    constexpr int AHEAD = 2;  // fragments are read two steps before their product
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      sa[k & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_frag(0, k), qf[k >> 1],
                                                          k < 2 ? zero : sa[k & 1], 0, 0, 0);
    // Scores of block b that the masks leave; only blocks on the edge of some row's range need it,
    // and mostly of one end: each bound by itself is a compare with a constant and a select a score.
    auto mask = [&](f16v* x, int b, int slot) {
      const int key0 = b * kCacheBlock;
      if (slot < 0 || key0 + kCacheBlock - 1 > wmin) {
        const int last = (slot < 0 ? -1 : pos - key0) - hf * 4;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[t][j] = t * 32 + (j >> 2) * 8 + (j & 3) > last ? kNegInf : x[t][j];
      }
      if (key0 <= below_window(wmax, A.window)) {
        const int first = low - key0 - hf * 4;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[t][j] = t * 32 + (j >> 2) * 8 + (j & 3) <= first ? kNegInf : x[t][j];
      }
    };
    mask(sa, b0, s0);
    float top = kNegInf;  // maximum of the block whose softmax is next
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, sa[t][j]);
    top = max_halves(top);
    __syncthreads();

    // Block b: sc its scores, sn the place of the next one's. One product a step; the fences
    // keep the VALU work spread between them (left alone, the compiler gathers it behind).
    auto iterate = [&](f16v* sc, f16v* sn, int b) {
      const int buf = (b - b0) & 1;
      bf16x8 kf[3], vf[3];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) kf[k] = k_frag(buf ^ 1, k);
      const int s3 = block_slot(C, table, b + 3 < b1 ? b + 3 : e);
      // The reference m of the weights is a whole number and moves only when the maximum outgrows
      // it by 2^8: weights up to 256 cost no precision, and in most blocks nothing is rescaled.
      const float want = ceilf(top * scale);
      const bool grows = want > m + 8.f;
      if (__any(grows)) {
        const float alpha = grows ? exp2_f(m - want) : 1.f;
        m = grows ? want : m;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < DT; ++i) o[i] *= alpha;
      }
      const float base = m == kNegInf ? 0.f : m;
      uint32_t pw[4][4];  // weights, 4 x 8 bf16
      constexpr int PAIRS = 16 / STEPS > 0 ? 16 / STEPS : 1;
      __builtin_amdgcn_sched_barrier(0);
      // K(b + 1) Q^T beside the softmax of b
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        if (k + AHEAD < STEPS) kf[(k + AHEAD) % 3] = k_frag(buf ^ 1, k + AHEAD);
        if (k + AHEAD >= STEPS) vf[k + AHEAD - STEPS] = v_frag(buf, k + AHEAD - STEPS);
        sn[k & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[k % 3], qf[k >> 1],
                                                            k < 2 ? zero : sn[k & 1], 0, 0, 0);
#pragma unroll
        for (int e2 = k * PAIRS; e2 < (k + 1) * PAIRS; ++e2) {
          const int t = e2 / 8, j = e2 % 8 * 2;
          const float x = exp2_f(fmaf(sc[t][j], scale, -base));
          const float y = exp2_f(fmaf(sc[t][j + 1], scale, -base));
          // One rounding of the weight to bf16 (at most 2^-8 of it), the matrix cores' type. The
          // sum is that of the rounded weights: what rounding takes from the numerator it then
          // takes from the denominator, all of it where one key holds most of the weight.
          const bf16x2 w2 = {static_cast<bf16>(x), static_cast<bf16>(y)};
          l = __builtin_amdgcn_fdot2_f32_bf16(w2, bf16x2{one, one}, l, false);
          pw[t * 2 + (j >> 3)][(j & 7) >> 1] = __builtin_bit_cast(uint32_t, w2);
          // (an empty statement that wants the pair here: it is not used before the branch below,
          // and would be computed behind it)
          asm volatile("" : "+v"(pw[t * 2 + (j >> 3)][(j & 7) >> 1]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      asm volatile("" : "+v"(l));
      mask(sn, b + 1, s1);
      bf16x8 pf[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        pf[u] = __builtin_bit_cast(bf16x8, make_uint4(pw[u][0], pw[u][1], pw[u][2], pw[u][3]));
      // V(b)^T P(b)^T beside the next maximum and the staging of K(b + 2) and V(b + 1)
      top = kNegInf;
#pragma unroll
      for (int v = 0; v < STEPS; ++v) {
        if (v + AHEAD < STEPS) vf[(v + AHEAD) % 3] = v_frag(buf, v + AHEAD);
        o[v % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[v % 3], pf[v / DT], o[v % DT], 0, 0, 0);
        if (v < NC) put_k(buf, v);
        if (v >= NC && v < 2 * NC) put_v(buf ^ 1, v - NC, s1);
        if (v == 2 * NC) {
          fetch_k(s3);  // K(b + 3), or the last block once more, unused
          fetch_v(s2);
        }
#pragma unroll
        for (int j = v * 32 / STEPS; j < (v + 1) * 32 / STEPS; ++j) top = fmaxf(top, sn[j >> 4][j & 15]);
        __builtin_amdgcn_sched_barrier(0);
      }
      top = max_halves(top);
      s0 = s1;
      s1 = s2;
      s2 = s3;
      __syncthreads();
    };
    for (int b = b0; b < b1; ++b) {
      iterate(sa, sb, b);
      if (++b >= b1) break;
      iterate(sb, sa, b);
    }
  }

  l += __shfl_xor(l, 32, 64);
  if (W.splits == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    // The rows pass through the wave's own part of LDS (nobody reads tiles there any more) and
    // leave in whole lines, past the caches, so that they are out before the kernel's end has to
    // write the caches back (8192 tokens, window 514, 16 heads on 8, when it was changed: 74 us as
    // they lie, in pieces of 16 bytes; 69 in lines; 66 in lines past the caches; now 55 to 61).
    constexpr int LR = D / 8, RP = 64 / LR;  // lanes of a row, rows of a pass
    bf16* const own = reinterpret_cast<bf16*>(&lds) + wave * 32 * KLD;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        bf16x8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<bf16>(o[i][j + e] * inv);
        *reinterpret_cast<bf16x8*>(own + col * KLD + i * 32 + j * 2 + hf * 8) = x;
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int p = 0; p < 32 / RP; ++p) {
      const int r2 = p * RP + lane / LR, ch = lane % LR * 8;
      const long to = __shfl((int)out, r2, 64);
      const bf16x8 x = *reinterpret_cast<const bf16x8*>(own + r2 * KLD + ch);
      if (wr0 + r2 < rows)
        __builtin_nontemporal_store(x, reinterpret_cast<bf16x8*>((bf16*)A.o + to * D + ch));
    }
  } else if (live) {
    if (hf == 0) {
      float* ml = W.ml + ((long)piece * W.rows + out) * 2;
      ml[0] = m;
      ml[1] = l;
    }
    if (l == 0.f) return;  // (the merge does not read this piece)
    float* dst = W.o + ((long)piece * W.rows + out) * D + hf * 8;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f4*>(dst + i * 32 + (j >> 1) * 16 + (j & 1) * 4) =
            f4{o[i][j * 4], o[i][j * 4 + 1], o[i][j * 4 + 2], o[i][j * 4 + 3]};
  }
}

// ---------------------------------------------------------------- merge of the pieces

// D / 4 lanes hold a row; SG such groups share a row's pieces (piece p to group p % SG) and are
// added in order. A piece without keys (sum 0) left no output. FEW: rows of the few-row kernel in a
// mixed batch, `few` for each (sequence, kv head); else the rows of the output, but for those that
// are marked as the few-row kernel's.
template <int D, int SG, bool FEW>
__global__ void __launch_bounds__(256) gdn2_cache_attn_merge_kernel(CacheAttnArgs A, Pieces W) {
  constexpr int LN = D / 4, RPB = 256 / LN / SG;
  const int l = threadIdx.x % LN, grp = threadIdx.x / LN, sg = grp % SG;
  const long row = (long)blockIdx.x * RPB + grp / SG;
  long out = row;  // row of the output
  if (row >= W.rows) return;  // (all lanes of a row, and with SG > 1 all of a workgroup)
  if (FEW) {
    const int r = (int)(row % W.few), G = A.Hq / A.Hk;
    const long nh = row / W.few;
    const int n = (int)(nh / A.Hk), h = (int)(nh % A.Hk);
    const int first = clamped_offset(A.c.cu_seqlens, n, A.c.T);
    const long rows = (long)(clamped_offset(A.c.cu_seqlens, n + 1, A.c.T) - first) * G;
    if (r >= rows || rows > W.few) return;
    out = ((long)first + r / G) * A.Hq + h * G + r % G;
  } else if (A.c.cu_seqlens != nullptr) {  // rows outside the sequences stay as they are
    const long tok = row / A.Hq;
    if (tok < clamped_offset(A.c.cu_seqlens, 0, A.c.T) ||
        tok >= clamped_offset(A.c.cu_seqlens, A.c.N, A.c.T) ||
        (W.few && W.ml[row * 2 + 1] < 0.f))
      return;
  }
  float top = kNegInf;
  for (int p = l; p < W.splits; p += LN) {
    const f2v ml = *reinterpret_cast<const f2v*>(W.ml + ((long)p * W.rows + row) * 2);
    if (ml[1] != 0.f) top = fmaxf(top, ml[0]);
  }
#pragma unroll
  for (int k = 1; k < LN; k <<= 1) top = fmaxf(top, __shfl_xor(top, k, 64));
  f4 acc = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int base = 0; base < W.splits; base += LN) {
    float f = 0.f, fl = 0.f;  // weight of piece base + l, and its share of the sum
    if (base + l < W.splits) {
      const f2v ml = *reinterpret_cast<const f2v*>(W.ml + ((long)(base + l) * W.rows + row) * 2);
      if (ml[1] != 0.f) {
        f = exp2_f(ml[0] - top);
        fl = ml[1] * f;
      }
    }
    const int n = W.splits - base < LN ? W.splits - base : LN;
#pragma unroll 4
    for (int j = sg; j < n; j += SG) {
      const float fj = __shfl(f, j, LN), lj = __shfl(fl, j, LN);
      const f4 x = *reinterpret_cast<const f4*>(W.o + ((long)(base + j) * W.rows + row) * D + l * 4);
      sum += lj;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += lj == 0.f ? 0.f : x[i] * fj;
    }
  }
  if constexpr (SG > 1) {
    __shared__ __align__(16) float red[256][4];
    __shared__ float rs[256 / LN];
    *reinterpret_cast<f4*>(red[threadIdx.x]) = acc;
    if (l == 0) rs[grp] = sum;
    __syncthreads();
    if (sg != 0) return;
#pragma unroll
    for (int j = 1; j < SG; ++j) {
      acc += *reinterpret_cast<const f4*>(red[threadIdx.x + j * LN]);
      sum += rs[grp + j];
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<bf16x4*>((bf16*)A.o + out * D + l * 4) =
      bf16x4{static_cast<bf16>(acc[0] * inv), static_cast<bf16>(acc[1] * inv),
             static_cast<bf16>(acc[2] * inv), static_cast<bf16>(acc[3] * inv)};
}

// Floats of one pass's partial results (`pieces` of each row: outputs, then maximum and sum), whole
// 16-byte pieces: the next pass's, read as vectors, lie behind them.
size_t partial_floats(int pieces, long rows, int d) {
  return ((size_t)pieces * rows * (d + 2) + 3) / 4 * 4;
}

template <int D>
hipError_t run_few(const CacheAttnArgs& a, int row_tiles, int waves, int split_blocks, const Pieces& w) {
  const hipStream_t st = (hipStream_t)a.stream;
  const dim3 grid((unsigned)((long)a.c.N * a.Hk * w.splits));
  if (row_tiles == 2)
    hipLaunchKernelGGL((gdn2_cache_attn_rows_kernel<D, 2, 4>), grid, dim3(256), 0, st, a, split_blocks, w);
  else if (waves == 8)
    hipLaunchKernelGGL((gdn2_cache_attn_rows_kernel<D, 1, 8>), grid, dim3(512), 0, st, a, split_blocks, w);
  else
    hipLaunchKernelGGL((gdn2_cache_attn_rows_kernel<D, 1, 4>), grid, dim3(256), 0, st, a, split_blocks, w);
  return hipGetLastError();
}

template <int D, bool FEW>
hipError_t run_merge(const CacheAttnArgs& a, const Pieces& w) {
  const hipStream_t st = (hipStream_t)a.stream;
  // Many pieces: a workgroup a row, or a row's chain of loads would be the call's latency
  // (129 pieces of 256 rows: 44 us with one group a row).
  constexpr int GR = 256 / (D / 4);
  if (w.splits > 8)
    hipLaunchKernelGGL((gdn2_cache_attn_merge_kernel<D, GR, FEW>), dim3((unsigned)w.rows), dim3(256),
                       0, st, a, w);
  else
    hipLaunchKernelGGL((gdn2_cache_attn_merge_kernel<D, 1, FEW>),
                       dim3((unsigned)((w.rows + GR - 1) / GR)), dim3(256), 0, st, a, w);
  return hipGetLastError();
}

template <int D>
hipError_t run(const CacheAttnArgs& a, const CacheAttnPlan& p) {
  const hipStream_t st = (hipStream_t)a.stream;
  const long tokens = a.c.cu_seqlens ? a.c.T : (long)a.c.N * a.c.T;
  Pieces w;
  w.rows = tokens * a.Hq;
  w.splits = p.splits;
  w.few = p.mixed_rows;
  w.o = (float*)a.workspace;
  w.ml = w.o + (size_t)p.splits * w.rows * D;
  hipError_t e;
  if (p.few_rows) {
    e = run_few<D>(a, p.row_tiles, p.waves, p.split_blocks, w);
  } else {
    const int units = a.c.cu_seqlens ? p.row_tiles : p.row_tiles * a.c.N;
    const dim3 grid((unsigned)((long)units * a.Hk * p.splits));
    if (D == 64 || p.tile_rows == 128)
      hipLaunchKernelGGL((gdn2_cache_attn_tile_kernel<D, 4>), grid, dim3(256), 0, st, a, units,
                         p.split_blocks, w);
    else
      hipLaunchKernelGGL((gdn2_cache_attn_tile_kernel<D, D == 64 ? 4 : 8>), grid, dim3(512), 0, st,
                         a, units, p.split_blocks, w);
    e = hipGetLastError();
  }
  if (e == hipSuccess && p.splits > 1) e = run_merge<D, false>(a, w);
  if (e != hipSuccess || p.mixed_rows == 0) return e;
  if (p.splits > 1) w.o += partial_floats(p.splits, w.rows, D);
  w.rows = (long)a.c.N * a.Hk * p.mixed_rows;
  w.splits = p.mixed_splits;
  w.ml = w.o + (size_t)p.mixed_splits * w.rows * D;
  e = run_few<D>(a, p.mixed_rows / 16, p.mixed_waves, p.mixed_blocks, w);
  if (e == hipSuccess && p.mixed_splits > 1) e = run_merge<D, true>(a, w);
  return e;
}

}  // namespace

CacheAttnPlan cache_attn_plan(bool packed, int N, int T, int Hq, int Hk, int d, int max_blocks,
                              int window) {
  CacheAttnPlan p;
  const long G = Hq / Hk, rows = T * G;
  // blocks that `tokens` new tokens of a sequence can reach: the table's, or what the window and
  // the tokens span
  const auto reach = [&](long tokens) {
    const long w = ((long)window + tokens + kCacheBlock - 3) / kCacheBlock + 1;
    return window > 0 && w < max_blocks ? w : (long)max_blocks;
  };
  const long nb = reach(T);
  // The few-row kernel's pieces. The lengths are on the device, so the cut goes by the table's
  // width: pieces past a sequence's end leave at once, and the others are as long as for a sequence
  // that fills the table (8 sequences of 4096 tokens, 8 kv heads: 16.7 us with a table of 64 blocks,
  // 21.7 of 128, 33.7 of 512).
  const auto cut = [&](long nb, int row_tiles, int& waves, int& split_blocks, int& splits) {
    const long groups = (long)N * Hk;
    // A workgroup a compute unit: twice or half as many pieces cost 15 to 25% (4 sequences of 32 K
    // tokens, 4 drafts, 16 heads on 2: 21.8 us; 25.0 with 512 workgroups, 27.5 with 128).
    long per = nb * groups / 256;
    if (per < nb / 256) per = nb / 256;
    per = (per + 3) / 4 * 4;  // a block a wave
    if (per < 4) per = 4;
    waves = 4;
    if (row_tiles == 1 && per < nb && nb <= 8) {
      // up to a block a wave in one workgroup of 8: no merge (512 tokens: 7.2 against 7.9 us; 16
      // blocks would take 10.3 against 9.0, a compute unit draws but 50 GB/s)
      waves = 8;
      per = nb;
    }
    split_blocks = (int)per;
    splits = (int)((nb + per - 1) / per);
    if (splits < 1) splits = 1;
  };
  p.few_rows = rows <= 32;
  p.tile_rows = p.waves = 0;
  p.mixed_rows = p.mixed_waves = p.mixed_blocks = 0;
  p.mixed_splits = 1;
  p.mixed_part_rows = 0;
  if (p.few_rows) {
    p.row_tiles = rows <= 16 ? 1 : 2;
    cut(nb, p.row_tiles, p.waves, p.split_blocks, p.splits);
  } else {
    auto tiles = [&](int r) { return packed ? rows / r + N : (rows + r - 1) / r * N; };
    // Pieces of the key axis where whole tiles would leave compute units idle, or one long tile would
    // be the call's time. By what was measured in us a block (of the longest tile; c1: a workgroup
    // alone on its unit, c2: two, unit: a unit's throughput), 5 us for the merge and 4 bytes a ps
    // over its partial rows: 512 tokens behind 7680, 16 heads on 4: 146 us whole, 55 in eight; 8
    // tokens over 32 K, 16 on 2: 624 and 24; 3000 tokens alone, 8 heads: 63 and 50 in two (d = 64: 50
    // and 37); but 2048 tokens alone, 16 on 4: 41 and 50 in two.
    const double c1 = d == 64 ? 0.92 : 1.25, c2 = d == 64 ? 1.31 : 2.0, unit = d == 64 ? 0.68 : 1.03;
    const long wgs = tiles(128) * Hk;
    // blocks of the longest tile, and of the mean one (prompts are causal)
    const long most = reach(127 / G + 2 < T ? 127 / G + 2 : T);
    const double own = (double)(packed ? T / N : T) / kCacheBlock;
    const double mean = window > 0 ? (double)most : most - 0.5 * (own < most ? own : (double)most);
    const auto cost = [&](long s) {
      const double per = (double)((most + s - 1) / s), work = (double)wgs * mean;
      const double chain = per * ((double)wgs * s * mean / most <= 256.0 ? c1 : c2);
      const double merge = s > 1 ? 5.0 + 2.0e-6 * d * (double)(rows * (packed ? 1 : N) * Hk) * s : 0.0;
      return (chain > work * unit / 256 ? chain : work * unit / 256) + merge;
    };
    long best = 1;
    // (Packed sequences differ in length, and the table's width says less of them: there only idle
    // units are filled. 64 single tokens 46 us with two pieces for the tiles as well, 38 without.)
    for (long s : {packed ? 1L : 2L, packed ? 1L : 3L, 256 / wgs, 512 / wgs}) {
      if (s > most / 4) s = most / 4;
      if (s > 1 && cost(s) < cost(best)) best = s;
    }
    const long per = best == 1 ? nb : (most + best - 1) / best;
    // Eight waves on one staged copy of K and V where there are tiles enough: 255 against 280 us
    // (8192 tokens, 16 heads on 4); but 48 against 45 us where a tile has only 9 blocks (8 x 1024
    // tokens, window 512; 23 against 16 of one sequence), and at d = 64 a block has only half as
    // much to stage as 512 threads take at once.
    p.tile_rows = best == 1 && d == 128 && most > 24 && tiles(256) * Hk >= 512 ? 256 : 128;
    p.row_tiles = (int)(packed ? tiles(p.tile_rows) : tiles(p.tile_rows) / N);
    p.split_blocks = (int)per;
    p.splits = best == 1 ? 1 : (int)((most + per - 1) / per);
    // Packed batches may hold single tokens and drafts beside prompts, and only the device knows
    // which. A tile for one token walks its whole context alone, so sequences of few rows get a pass
    // of the few-row kernel: 64 single tokens of 2 K to 4 K tokens, 16 heads on 4: 104 us as tiles,
    // 38 with the pass; one over 32 K tokens beside a prompt of 2048: 670 and 61. It costs 3 us
    // where all are prompts, and a tile of 32 blocks 35 us: so not below that, unless the
    // sequences' tiles alone would fill the card (128 tokens over 1024 beside a prompt: 51 and 41).
    if (packed && N > 1 && G <= 32) {
      const int few = G <= 8 ? 16 : 32;
      const long nf = reach(few / G);
      if (nf >= 32 || (long)N * Hk >= 512) {
        p.mixed_rows = few;
        cut(nf, few / 16, p.mixed_waves, p.mixed_blocks, p.mixed_splits);
        p.mixed_part_rows = (long)N * Hk * few;
      }
    }
  }
  if (p.splits < 1) p.splits = 1;
  return p;
}

size_t cache_attn_workspace_bytes(const CacheAttnPlan& p, long tokens, int Hq, int d) {
  size_t floats = 0;
  if (p.splits > 1) floats += partial_floats(p.splits, tokens * Hq, d);
  if (p.mixed_splits > 1) floats += partial_floats(p.mixed_splits, p.mixed_part_rows, d);
  return floats * sizeof(float);
}

long cache_attn_groups(const CacheAttnPlan& p, bool packed, int N, int Hk) {
  const long units = p.few_rows ? N : packed ? p.row_tiles : (long)p.row_tiles * N;
  const long tiles = units * Hk * p.splits, mixed = p.mixed_rows ? (long)N * Hk * p.mixed_splits : 0;
  return tiles > mixed ? tiles : mixed;
}

hipError_t launch_cache_attn(const CacheAttnArgs& a, const CacheAttnPlan& p) {
  return a.d == 64 ? run<64>(a, p) : run<128>(a, p);
}

}  // namespace gdn2
