// Rows of queries and keys on gfx950: the norm of each head and the position rotation in one
// pass (forward, backward), and the serving prologue that also writes keys and values into the
// paged 8-bit cache.
//
// One head row x of d channels, weight w, position p, frequencies f:
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x w
//   pair i < rot / 2, (a, b) = (n[i], n[i + rot / 2]) or (n[2i], n[2i + 1]):
//     y_a = a cos(p f_i) - b sin(p f_i),  y_b = b cos(p f_i) + a sin(p f_i);  the rest as n
// and its gradient, with dn the rotation of dy by -p f:
//   dw = sum over rows of dn x r,  dx = r (w dn - x (r^2 / d) sum_c(w dn x))
// Everything is fp32 from the load to the one rounding at the store; the angle is fp64 up to
// the fraction of a quarter turn, since p f reaches 10^6 turns where fp32 has lost the fraction.
//
// All of it is bound by memory: each row is read once and written once. A row lies on d / 8
// lanes, 8 channels a lane, so that every lane holds whole pairs and the rotation needs no
// exchange: a lane has 4 pairs, loaded as two 4-channel pieces (the members half a rotation
// apart) or as 8 neighbouring channels. A wave takes one token and up to 4 rows per lane group
// of it, which share the token's sines.

#include "gdn2_attn_device.h"

namespace gdn2 {

namespace {

constexpr int kRowsPerLane = 4;  // rows in flight per lane group: 16 heads a wave at d = 128
constexpr int kBwdGroups = 512;  // workgroups along the tokens in the backward

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Piece4;
template <> struct Piece4<bf16> {
  bf16x4 r;
  __device__ void load(const bf16* p) { r = *reinterpret_cast<const bf16x4*>(p); }
  __device__ float get(int i) const { return static_cast<float>(r[i]); }
};
template <> struct Piece4<float> {
  f4 r;
  __device__ void load(const float* p) { r = *reinterpret_cast<const f4*>(p); }
  __device__ float get(int i) const { return r[i]; }
};
// Outputs go past the caches: a kernel's end would have to write them back (training forward 50.5 ->
// 46.1 us, the prologue of 8192 tokens 24.2 -> 22.3, with the attention behind it 296 -> 292).
__device__ __forceinline__ void store4(bf16* p, const float* f) {
  const bf16x4 v = {static_cast<bf16>(f[0]), static_cast<bf16>(f[1]), static_cast<bf16>(f[2]),
                    static_cast<bf16>(f[3])};
  __builtin_nontemporal_store(v, reinterpret_cast<bf16x4*>(p));
}
__device__ __forceinline__ void store4(float* p, const float* f) {
  __builtin_nontemporal_store(f4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f4*>(p));
}

// sin and cos of t quarter turns: the nearest whole number leaves in the low bits of t + 1.5 * 2^52
// (|t| < 2^51), the rest is exact in fp64; then the series on [-pi/4, pi/4] (the first omitted
// terms are 1.8e-9 and 2.5e-8, below fp32's rounding).
__device__ __forceinline__ void sincos_quarters(double t, float& s, float& c) {
  const double magic = 6755399441055744.0;  // 1.5 * 2^52
  const double w = t + magic;
  const int q = (int)(uint32_t)__double_as_longlong(w);
  const float x = static_cast<float>(t - (w - magic)) * 1.57079632679489661923f;
  const float y = x * x;
  const float sp =
      x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880))));
  const float cp = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320))));
  s = (q & 1) ? cp : sp;
  c = (q & 1) ? sp : cp;
  if (q & 2) s = -s;
  if ((q + 1) & 2) c = -c;
}

// A lane's share of a row: offsets of its two 4-channel pieces, and its 4 pairs (a, b) in them.
template <int D, bool IL>
struct Lane {
  int o0, o1;
  int pair;      // first pair
  bool rotated;  // rot % 8 == 0, so a lane's pairs are rotated together or not at all
  __device__ Lane(int l, int rot) {
    pair = 4 * l;
    rotated = pair < rot / 2;
    if (IL) {
      o0 = 8 * l;
      o1 = o0 + 4;
    } else if (rotated) {
      o0 = pair;
      o1 = pair + rot / 2;
    } else {  // channels past the rotation pass through, as two halves
      o0 = rot + pair - rot / 2;
      o1 = o0 + (D - rot) / 2;
    }
  }
};
template <bool IL, typename P>
__device__ __forceinline__ void to_pairs(const P& p0, const P& p1, float* a, float* b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = IL ? (i < 2 ? p0.get(2 * i) : p1.get(2 * i - 4)) : p0.get(i);
    b[i] = IL ? (i < 2 ? p0.get(2 * i + 1) : p1.get(2 * i - 3)) : p1.get(i);
  }
}
template <bool IL>
__device__ __forceinline__ void from_pairs(const float* a, const float* b, float* f0, float* f1) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f0[i] = IL ? ((i & 1) ? b[i / 2] : a[i / 2]) : a[i];
    f1[i] = IL ? ((i & 1) ? b[2 + i / 2] : a[2 + i / 2]) : b[i];
  }
}

// The 4 frequencies of a lane in quarter turns per position, 0 where it does not rotate (then the
// sines are 0 and the cosines 1).
template <int D, bool IL>
__device__ __forceinline__ void lane_freq(const Lane<D, IL>& L, const float* inv_freq, double* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = L.rotated ? static_cast<double>(inv_freq[L.pair + i]) * 0.63661977236758134308 : 0.0;
}

template <bool IL, int D>
__device__ __forceinline__ void lane_weight(const Lane<D, IL>& L, const float* w, float* wa,
                                            float* wb) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) wa[i] = wb[i] = 1.f;
    return;
  }
  Piece4<float> p0, p1;
  p0.load(w + L.o0);
  p1.load(w + L.o1);
  to_pairs<IL>(p0, p1, wa, wb);
}

// a, b: norm, weight and rotation in place.
template <int LANES, int D>
__device__ __forceinline__ void norm_rotate(float* a, float* b, const float* wa, const float* wb,
                                            const float* sn, const float* cs, bool norm,
                                            float eps) {
  float r = 1.f;
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += a[i] * a[i] + b[i] * b[i];
    r = rsqrtf(row_sum<LANES>(ss) * (1.f / D) + eps);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float na = a[i] * r * wa[i], nb = b[i] * r * wb[i];
    a[i] = na * cs[i] - nb * sn[i];
    b[i] = nb * cs[i] + na * sn[i];
  }
}

// Rows [0, nh) of one token: x -> y, both at the token's first row. One wave. place(pos) gives the
// token's position, after the rows' loads are out; where it returns false there is nothing to do
// (it may have written the rows itself).
template <typename T, int D, bool IL, typename F>
__device__ __forceinline__ void token_rows(const T* x, T* y, int nh, const float* inv_freq,
                                           const float* weight, int rot, bool norm, float eps,
                                           F place) {
  constexpr int LANES = D / 8, RPW = 64 / LANES;
  const int lane = threadIdx.x & 63, grp = lane / LANES;
  const Lane<D, IL> L(lane % LANES, rot);
  Piece4<T> p0[kRowsPerLane], p1[kRowsPerLane];
#pragma unroll
  for (int u = 0; u < kRowsPerLane; ++u) {
    if (u * RPW >= nh) break;
    const int row = u * RPW + grp < nh ? u * RPW + grp : nh - 1;
    p0[u].load(x + (long)row * D + L.o0);
    p1[u].load(x + (long)row * D + L.o1);
  }
  double f[4];
  float wa[4], wb[4], sn[4], cs[4];
  lane_freq(L, inv_freq, f);
  lane_weight<IL>(L, weight, wa, wb);
  long pos;
  if (!place(pos)) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) sincos_quarters(f[i] * static_cast<double>(pos), sn[i], cs[i]);
#pragma unroll
  for (int u = 0; u < kRowsPerLane; ++u) {
    if (u * RPW >= nh) break;
    float a[4], b[4], f0[4], f1[4];
    to_pairs<IL>(p0[u], p1[u], a, b);
    norm_rotate<LANES, D>(a, b, wa, wb, sn, cs, norm, eps);
    from_pairs<IL>(a, b, f0, f1);
    const int row = u * RPW + grp;
    if (row < nh) {
      store4(y + (long)row * D + L.o0, f0);
      store4(y + (long)row * D + L.o1, f1);
    }
  }
}

template <int D> __host__ __device__ constexpr int heads_per_wave() {
  return 64 / (D / 8) * kRowsPerLane;
}

// grid (tokens / 4, chunks of heads: the queries', then the keys'); one wave a token.
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(256) gdn2_norm_rope_kernel(NormRopeArgs A) {
  constexpr int CH = heads_per_wave<D>();
  const long tok = (long)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (tok >= A.tokens) return;
  const int cq = (A.Hq + CH - 1) / CH;
  const bool isq = (int)blockIdx.y < cq;
  const int h0 = (isq ? blockIdx.y : blockIdx.y - cq) * CH;
  const int H = isq ? A.Hq : A.Hk;
  const int nh = H - h0 < CH ? H - h0 : CH;
  const T* x = (const T*)(isq ? A.q : A.k) + tok * (isq ? A.q_stride : A.k_stride) + (long)h0 * D;
  T* y = (T*)(isq ? A.q_out : A.k_out) + (tok * H + h0) * D;
  token_rows<T, D, IL>(x, y, nh, A.inv_freq, isq ? A.q_weight : A.k_weight, A.rot, A.norm,
                             A.eps, [&](long& pos) {
    pos = A.positions ? A.positions[tok] : tok % A.T;
    return true;
  });
}

// Backward. grid (groups, chunks): a wave walks tokens and keeps its channels' weight gradient
// in registers; the workgroup leaves one partial row [D] in the workspace, summed in order by
// the second kernel (no atomics: the same inputs give the same bits).
template <typename T, int D, bool IL>
__global__ void __launch_bounds__(256) gdn2_norm_rope_bwd_kernel(NormRopeArgs A) {
  constexpr int CH = heads_per_wave<D>(), LANES = D / 8, RPW = 64 / LANES;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grp = lane / LANES;
  const int cq = (A.Hq + CH - 1) / CH;
  const bool isq = (int)blockIdx.y < cq;
  const int h0 = (isq ? blockIdx.y : blockIdx.y - cq) * CH;
  const int H = isq ? A.Hq : A.Hk;
  const int nh = H - h0 < CH ? H - h0 : CH;
  const T* xb = (const T*)(isq ? A.q : A.k) + (long)h0 * D;
  const T* gb = (const T*)(isq ? A.gq : A.gk) + (long)h0 * D;
  T* yb = (T*)(isq ? A.q_out : A.k_out) + (long)h0 * D;
  const long xs = isq ? A.q_stride : A.k_stride;
  const Lane<D, IL> L(lane % LANES, A.rot);
  double f[4];
  float wa[4], wb[4], da[4] = {}, db[4] = {};
  lane_freq(L, A.inv_freq, f);
  lane_weight<IL>(L, isq ? A.q_weight : A.k_weight, wa, wb);
  for (long tok = (long)blockIdx.x * 4 + wave; tok < A.tokens; tok += (long)gridDim.x * 4) {
    Piece4<T> x0[kRowsPerLane], x1[kRowsPerLane], g0[kRowsPerLane], g1[kRowsPerLane];
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      if (u * RPW >= nh) break;
      const long row = u * RPW + grp < nh ? u * RPW + grp : nh - 1;
      x0[u].load(xb + tok * xs + row * D + L.o0);
      x1[u].load(xb + tok * xs + row * D + L.o1);
      g0[u].load(gb + (tok * H + row) * D + L.o0);
      g1[u].load(gb + (tok * H + row) * D + L.o1);
    }
    const long pos = A.positions ? A.positions[tok] : tok % A.T;
    float sn[4], cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sincos_quarters(f[i] * static_cast<double>(pos), sn[i], cs[i]);
#pragma unroll
    for (int u = 0; u < kRowsPerLane; ++u) {
      if (u * RPW >= nh) break;
      float a[4], b[4], ga[4], gb_[4], f0[4], f1[4];
      to_pairs<IL>(x0[u], x1[u], a, b);
      to_pairs<IL>(g0[u], g1[u], ga, gb_);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float na = ga[i] * cs[i] + gb_[i] * sn[i];
        const float nb = gb_[i] * cs[i] - ga[i] * sn[i];
        ga[i] = na;
        gb_[i] = nb;
        ss += a[i] * a[i] + b[i] * b[i];
        dot += wa[i] * na * a[i] + wb[i] * nb * b[i];
      }
      float r = 1.f, back = 0.f;
      if (A.norm) {
        ss = row_sum<LANES>(ss);
        dot = row_sum<LANES>(dot);
        r = rsqrtf(ss * (1.f / D) + A.eps);
        back = r * r * (1.f / D) * dot;
      }
      const int row = u * RPW + grp;
      const bool live = row < nh;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        da[i] += live ? ga[i] * a[i] * r : 0.f;
        db[i] += live ? gb_[i] * b[i] * r : 0.f;
        a[i] = r * (wa[i] * ga[i] - a[i] * back);
        b[i] = r * (wb[i] * gb_[i] - b[i] * back);
      }
      from_pairs<IL>(a, b, f0, f1);
      if (live) {
        store4(yb + (tok * H + row) * D + L.o0, f0);
        store4(yb + (tok * H + row) * D + L.o1, f1);
      }
    }
  }
  if (A.partial == nullptr) return;
  __shared__ float red[4][D];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int m = LANES; m < 64; m <<= 1) {
      da[i] += __shfl_xor(da[i], m, 64);
      db[i] += __shfl_xor(db[i], m, 64);
    }
  }
  if (grp == 0) {
    float f0[4], f1[4];
    from_pairs<IL>(da, db, f0, f1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      red[wave][L.o0 + i] = f0[i];
      red[wave][L.o1 + i] = f1[i];
    }
  }
  __syncthreads();
  float* out = A.partial + ((long)blockIdx.y * gridDim.x + blockIdx.x) * D;
  for (int c = threadIdx.x; c < D; c += 256)
    out[c] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
}

// Sum of the partial rows in fp64. grid (2, D / 16): queries, keys; 16 columns x 64 rows of
// threads.
template <int D>
__global__ void __launch_bounds__(1024)
gdn2_weight_grad_kernel(const float* partial, long rows_q, long rows_k, float* dwq, float* dwk) {
  __shared__ double red[64][17];
  float* out = blockIdx.x == 0 ? dwq : dwk;
  if (out == nullptr) return;
  const float* p = partial + (blockIdx.x == 0 ? 0 : rows_q * D);
  const long rows = blockIdx.x == 0 ? rows_q : rows_k;
  const int c = threadIdx.x & 15, j = threadIdx.x >> 4;
  p += blockIdx.y * 16 + c;
  double acc[4] = {};  // four loads in flight a thread: a chain of single ones is all latency
  for (long r = j; r < rows; r += 256) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = r + i * 64 < rows ? p[(r + i * 64) * D] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += x[i];
  }
  red[j][c] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
  __syncthreads();
  for (int half = 32; half > 0; half >>= 1) {
    if (j < half) red[j][c] += red[j + half][c];
    __syncthreads();
  }
  if (j == 0) out[blockIdx.y * 16 + c] = static_cast<float>(red[0][c]);
}

// ------------------------------------------------------------------ the 8-bit cache

// Smallest power of two s >= 2^-64 with amax <= 448 s (448: the largest e4m3). A power of two
// costs a floating-point code no precision, makes the value e4m3 * s exact in bf16, and lets a
// block's scale grow later by shifting exponents.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  if (e < -64) e = -64;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
__device__ __forceinline__ uint32_t rescale_fp8(uint32_t x, float f) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)x, true);
  return pack_fp8(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}
__device__ __forceinline__ uint4 rescale_fp8(uint4 x, float f) {
  return make_uint4(rescale_fp8(x.x, f), rescale_fp8(x.y, f), rescale_fp8(x.z, f),
                    rescale_fp8(x.w, f));
}

// Below 248 * 2^120, from where on a code would stand for 2^128; false for NaN and infinities.
__device__ __forceinline__ bool storable(float x) {
  return (__float_as_uint(x) & 0x7fffffffu) < 0x7f780000u;
}

// Column of token t in a value block: the order in which a lane of the attention kernels'
// 16x16 tiles holds the keys (4 tokens of each of the 4 key tiles), so that a lane's share of a
// value row is 16 contiguous bytes.
__host__ __device__ constexpr int value_column(int t) {
  return ((t >> 2) & 3) * 16 + (t >> 4) * 4 + (t & 3);
}

// Serving prologue. Workgroups [0, kv_groups): one (sequence, cache block that new tokens
// touch, kv head) each: norm and rotation of the block's new keys, the block's scales, codes
// into the cache. The rest: query rows, a wave a token and chunk of heads (behind the longer
// work: 28 against 33 us for 10 K tokens of prompts with the query rows in front).
//
// A (block, head) has one writer, so a growing scale needs no exchange with another workgroup.
// Rows of a block are dealt so that a lane group holds 4 neighbouring tokens (2 at d = 64):
// their codes of one value channel are neighbouring bytes of the block. FEW: as many new tokens at
// most as a wave has lane groups, and a wave a (block, head): a single token has work for 16 lanes,
// and what bounds it is how many of these chains of loads are under way (one token of 256 sequences,
// 4 heads: 10.0 us with four waves, 7.8 with one; of 512, 16 heads: 36.7 and 20.5).
template <int D, bool IL, bool FEW>
__global__ void __launch_bounds__(FEW ? 64 : 256, 5)
gdn2_attn_prologue_kernel(AttnPrologueArgs A, int kv_groups, int units_per_seq) {
  typedef bf16 T;
  constexpr int NT = FEW ? 64 : 256, NW = NT / 64;
  constexpr int LANES = D / 8, PASSES = FEW ? 1 : kCacheBlock / (NT / LANES);
  const CacheView& C = A.c;
  if ((int)blockIdx.x >= kv_groups) {
    constexpr int CH = heads_per_wave<D>();
    const int chunks = (A.Hq + CH - 1) / CH;
    const long item = (long)((int)blockIdx.x - kv_groups) * NW + (threadIdx.x >> 6);
    const int tok = __builtin_amdgcn_readfirstlane((int)(item / chunks));
    const int tokens = C.cu_seqlens ? C.T : C.N * C.T;
    if (tok >= tokens) return;
    const int h0 = (int)(item % chunks) * CH;
    const int nh = A.Hq - h0 < CH ? A.Hq - h0 : CH;
    T* y = (T*)A.q_out + ((long)tok * A.Hq + h0) * D;
    token_rows<T, D, IL>((const T*)A.q + tok * A.q_stride + (long)h0 * D, y, nh, A.inv_freq,
                                A.q_weight, A.rot, A.norm, A.eps, [&](long& pos) {
      SeqSpan s;
      if (C.cu_seqlens == nullptr) s = seq_span(C, tok / C.T);
      else packed_span(C, tok, s, [](int first, int) { return (long)first; });
      if (tok < s.first || tok >= s.first + s.count) return false;  // behind the last sequence
      pos = s.len - s.count + (tok - s.first);
      if (pos >= 0) return true;
      for (int c = threadIdx.x & 63; c < nh * (D / 8); c += 64)  // no token there
        reinterpret_cast<uint4*>(y)[c] = make_uint4(0, 0, 0, 0);
      return false;
    });
    return;
  }

  const int unit = blockIdx.x / A.Hk, h = blockIdx.x % A.Hk;
  int n, x;
  SeqSpan s;
  if (C.cu_seqlens == nullptr) {
    n = unit / units_per_seq;
    x = unit % units_per_seq;
    s = seq_span(C, n);
  } else {  // sequence n owns the units from floor(first row / 64) + 2 n on
    n = packed_span(C, unit, s, [](int first, int i) { return (long)first / kCacheBlock + 2L * i; });
    x = unit - s.first / kCacheBlock - 2 * n;
    if (x < 0) return;
  }
  n = uniform(n);
  x = uniform(x);
  s = uniform(s);
  const long start = s.len - s.count;                       // position of the first new row
  const long first = start < 0 ? 0 : start;                 // position of the first new token
  const long blk = first / kCacheBlock + x;
  if (blk * kCacheBlock >= s.len || blk >= C.max_blocks) return;
  // new rows of this block: offsets [r0, r1)
  const int r0 = first > blk * kCacheBlock ? (int)(first - blk * kCacheBlock) : 0;
  const int r1 = s.len - blk * kCacheBlock < kCacheBlock ? (int)(s.len - blk * kCacheBlock)
                                                         : kCacheBlock;
  if (r0 >= r1) return;  // no new token in it
  // A block of few new tokens is one wave's also where the launch could not know it, in a packed
  // batch: the others leave, whole waves that the barriers then do not wait for (512 single
  // tokens, 16 heads: 62.8 and 38.0 us; prompts 1% slower).
  const bool few = FEW || r1 - r0 <= 64 / LANES;
  if (few && threadIdx.x >= 64) return;
  const int nt = few ? 64 : NT;  // threads left
  const long row_of = s.first + (blk * kCacheBlock - start);  // token row of offset 0

  // The rows do not wait for the table: both loads go out together.
  const int tid = threadIdx.x, lane = tid & 63, grp = tid / LANES, l = tid % LANES;
  const Lane<D, IL> L(l, A.rot);
  Piece4<T> p0[PASSES], p1[PASSES];
  bf16x8 vr[PASSES];
  bool live[PASSES];
  const int own = few ? r0 + grp : grp * PASSES;  // first row of the lane group
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    const int r = own + u;
    live[u] = r >= r0 && r < r1 && (u == 0 || !few);
    const long row = row_of + (live[u] ? r : r0);
    const T* kr = (const T*)A.k + row * A.k_stride + (long)h * D;
    p0[u].load(kr + L.o0);
    p1[u].load(kr + L.o1);
    vr[u] = *reinterpret_cast<const bf16x8*>((const T*)A.v + row * A.v_stride + (long)h * D + 8 * l);
  }
  const int slot = scalar_load(C.block_table, (long)n * C.max_blocks + blk);
  if (slot < 0 || slot >= C.P) return;
  const long head = (long)slot * A.Hk + h;
  uint8_t* kc = C.k + head * (kCacheBlock * D);
  uint8_t* vc = C.v + head * (kCacheBlock * D);
  const bool older = r0 > 0;  // older tokens in the block
  const float ks_old = older ? C.k_scale[head] : 0.f, vs_old = older ? C.v_scale[head] : 0.f;

  double f[4];
  float wa[4], wb[4];
  lane_freq(L, A.inv_freq, f);
  lane_weight<IL>(L, A.k_weight, wa, wb);
  float ka[PASSES][4], kb[PASSES][4];
  bool fine[PASSES];
  float kmax = 0.f, vmax = 0.f;
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    fine[u] = true;
    if (!__any(live[u])) continue;  // a decoded token needs one pass of one wave
    float sn[4], cs[4];
    const double pos = static_cast<double>(blk * kCacheBlock + own + u);
#pragma unroll
    for (int i = 0; i < 4; ++i) sincos_quarters(f[i] * pos, sn[i], cs[i]);
    to_pairs<IL>(p0[u], p1[u], ka[u], kb[u]);
    norm_rotate<LANES, D>(ka[u], kb[u], wa, wb, sn, cs, A.norm, A.eps);
    float km = 0.f, vm = 0.f;
    int bad = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad |= !storable(ka[u][i]) | !storable(kb[u][i]);
      km = fmaxf(km, fmaxf(fabsf(ka[u][i]), fabsf(kb[u][i])));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float vf = static_cast<float>(vr[u][i]);
      bad |= !storable(vf);
      vm = fmaxf(vm, fabsf(vf));
    }
    const uint64_t all = __ballot(bad);  // a row is fine where none of its lanes saw something
    fine[u] = ((all >> (lane & ~(LANES - 1))) & ((1u << LANES) - 1)) == 0;
    if (live[u] && fine[u]) {
      kmax = fmaxf(kmax, km);
      vmax = fmaxf(vmax, vm);
    }
  }
  kmax = wave_max(kmax);
  vmax = wave_max(vmax);
  __shared__ float red[2][NW];
  __shared__ __align__(16) uint8_t vl[D * kCacheBlock];
  // Byte of (channel, column): the 16-byte chunk is swapped by the channel's octet, as the lanes
  // of a row write channels 8 apart.
  auto vplace = [](int ch, int col) {
    return ch * kCacheBlock + ((((col >> 4) ^ (ch >> 3)) & 3) << 4) + (col & 15);
  };
  if (lane == 0) {
    red[0][tid >> 6] = kmax;
    red[1][tid >> 6] = vmax;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < (few ? 1 : NW); ++w) {
    kmax = fmaxf(kmax, red[0][w]);
    vmax = fmaxf(vmax, red[1][w]);
  }
  const float ks = fmaxf(ks_old, block_scale(kmax)), vs = fmaxf(vs_old, block_scale(vmax));
  if (tid == 0) {  // every thread has read the old scales (the barrier above)
    C.k_scale[head] = ks;
    C.v_scale[head] = vs;
  }
  const float ki = 1.f / ks, vi = 1.f / vs;

  // keys: older rows follow a grown scale, new rows are written
  if (older && ks > ks_old)
    for (int c = tid; c < r0 * (D / 16); c += nt) {
      uint4* p = reinterpret_cast<uint4*>(kc) + c;
      *p = rescale_fp8(*p, ks_old * ki);
    }
  uint32_t vcode[PASSES][2];
#pragma unroll
  for (int u = 0; u < PASSES; ++u) {
    if (!__any(live[u])) continue;
    float f0[4], f1[4], v[8];
    from_pairs<IL>(ka[u], kb[u], f0, f1);
    // A key or value that cannot be stored marks its token: a key row of NaN, so that every query
    // that attends to it comes out NaN, and zeros as its value, so that queries that do not see
    // it are left alone.
    const uint32_t c0 =
        fine[u] ? pack_fp8(f0[0] * ki, f0[1] * ki, f0[2] * ki, f0[3] * ki) : 0x7f7f7f7fu;
    const uint32_t c1 =
        fine[u] ? pack_fp8(f1[0] * ki, f1[1] * ki, f1[2] * ki, f1[3] * ki) : 0x7f7f7f7fu;
    if (live[u]) {
      uint8_t* kr = kc + (own + u) * D;
      *reinterpret_cast<uint32_t*>(kr + L.o0) = c0;
      *reinterpret_cast<uint32_t*>(kr + L.o1) = c1;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fine[u] ? static_cast<float>(vr[u][i]) * vi : 0.f;
    vcode[u][0] = pack_fp8(v[0], v[1], v[2], v[3]);
    vcode[u][1] = pack_fp8(v[4], v[5], v[6], v[7]);
  }

  // values: few tokens into an unchanged block go out as single bytes; otherwise the whole
  // block is put together in LDS (older codes, new ones, zeros behind them in a block that
  // begins here: masked positions of the block then hold finite values) and written as rows.
  const bool vgrow = older && vs > vs_old;
  if (older && !vgrow && r1 - r0 <= 8) {
#pragma unroll
    for (int u = 0; u < PASSES; ++u)
      if (live[u]) {
        const int col = value_column(own + u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          vc[(8 * l + i) * kCacheBlock + col] = (uint8_t)(vcode[u][i >> 2] >> (8 * (i & 3)));
      }
    return;
  }
  for (int c = tid; c < D * 4; c += nt) {
    uint4 o = make_uint4(0, 0, 0, 0);
    if (older) o = reinterpret_cast<const uint4*>(vc)[c];
    if (vgrow) {  // the older tokens' codes, not what lies behind the last token (dropped drafts),
                  // unless the scale is now the largest: a code there could stand for infinity
      const uint32_t behind = vs < 0x1p120f ? ~0u : 0u;
      uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int left = r0 - (t * 16 + (c & 3) * 4);  // older tokens from this word's first on
        const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1;
        w[t] = (rescale_fp8(w[t], vs_old * vi) & keep) | (w[t] & ~keep & behind);
      }
      o = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(&vl[vplace(c >> 2, (c & 3) * 16)]) = o;
  }
  __syncthreads();
  bool whole = !few;
#pragma unroll
  for (int u = 0; u < PASSES; ++u) whole = whole && live[u];
  if (whole) {
    const int col = value_column(own);
#pragma unroll
    for (int k = 0; k < 2 && !FEW; ++k) {  // channels 8 l + 4 k ..: a transpose of 4 x PASSES bytes
      const uint32_t lo = __builtin_amdgcn_perm(vcode[PASSES > 1][k], vcode[0][k], 0x05010400u);
      const uint32_t hi = __builtin_amdgcn_perm(vcode[PASSES > 1][k], vcode[0][k], 0x07030602u);
      const int ch = 8 * l + 4 * k;
      if constexpr (PASSES == 4) {
        const uint32_t lo2 = __builtin_amdgcn_perm(vcode[3][k], vcode[2][k], 0x05010400u);
        const uint32_t hi2 = __builtin_amdgcn_perm(vcode[3][k], vcode[2][k], 0x07030602u);
        const uint32_t w[4] = {__builtin_amdgcn_perm(lo2, lo, 0x05040100u),
                               __builtin_amdgcn_perm(lo2, lo, 0x07060302u),
                               __builtin_amdgcn_perm(hi2, hi, 0x05040100u),
                               __builtin_amdgcn_perm(hi2, hi, 0x07060302u)};
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(&vl[vplace(ch + i, col)]) = w[i];
      } else {
        const uint32_t w[4] = {lo, lo >> 16, hi, hi >> 16};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint16_t*>(&vl[vplace(ch + i, col)]) = (uint16_t)w[i];
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < PASSES; ++u)
      if (live[u]) {
        const int col = value_column(own + u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          vl[vplace(8 * l + i, col)] = (uint8_t)(vcode[u][i >> 2] >> (8 * (i & 3)));
      }
  }
  __syncthreads();
  for (int c = tid; c < D * 4; c += nt)
    __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(&vl[vplace(c >> 2, (c & 3) * 16)]),
                                reinterpret_cast<u32x4*>(vc) + c);
}

// Units (sequence, touched cache block) and workgroups of query rows of the serving prologue.
struct PrologueGrid {
  bool few;  // one wave a (block, head)
  int per_seq;
  long units, q_groups;
};
PrologueGrid prologue_grid(const AttnPrologueArgs& a) {
  const int CH = a.d == 64 ? heads_per_wave<64>() : heads_per_wave<128>();
  const bool packed = a.c.cu_seqlens != nullptr;
  const long tokens = packed ? a.c.T : (long)a.c.N * a.c.T;
  PrologueGrid g;
  // blocks that T tokens can touch: 1 for one token, up to two partial ones around whole ones
  g.per_seq = packed ? 0 : (int)(((long)a.c.T + kCacheBlock - 2) / kCacheBlock + 1);
  g.units = packed ? a.c.T / kCacheBlock + 2L * a.c.N : (long)a.c.N * g.per_seq;
  g.few = !packed && a.c.T <= 64 / (a.d / 8);
  const long items = tokens * ((a.Hq + CH - 1) / CH);
  g.q_groups = g.few ? items : (items + 3) / 4;
  return g;
}

template <typename T, int D, bool IL>
hipError_t run_norm_rope(const NormRopeArgs& a) {
  constexpr int CH = heads_per_wave<D>();
  const int chunks = (a.Hq + CH - 1) / CH + (a.Hk + CH - 1) / CH;
  hipLaunchKernelGGL((gdn2_norm_rope_kernel<T, D, IL>),
                     dim3((unsigned)((a.tokens + 3) / 4), chunks), dim3(256), 0,
                     (hipStream_t)a.stream, a);
  return hipGetLastError();
}

template <typename T, int D, bool IL>
hipError_t run_norm_rope_bwd(const NormRopeArgs& a) {
  constexpr int CH = heads_per_wave<D>();
  const int cq = (a.Hq + CH - 1) / CH, ck = (a.Hk + CH - 1) / CH;
  const int groups = norm_rope_bwd_groups(a.tokens);
  hipLaunchKernelGGL((gdn2_norm_rope_bwd_kernel<T, D, IL>), dim3(groups, cq + ck), dim3(256), 0,
                     (hipStream_t)a.stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.partial == nullptr) return e;
  hipLaunchKernelGGL((gdn2_weight_grad_kernel<D>), dim3(2, D / 16), dim3(1024), 0,
                     (hipStream_t)a.stream, a.partial, (long)cq * groups, (long)ck * groups,
                     a.dq_weight, a.dk_weight);
  return hipGetLastError();
}

template <int D, bool IL>
hipError_t run_prologue(const AttnPrologueArgs& a) {
  const PrologueGrid g = prologue_grid(a);
  const int kv_groups = (int)(g.units * a.Hk);
  const dim3 grid((unsigned)(kv_groups + g.q_groups));
  if (g.few)
    hipLaunchKernelGGL((gdn2_attn_prologue_kernel<D, IL, true>), grid, dim3(64), 0,
                       (hipStream_t)a.stream, a, kv_groups, g.per_seq);
  else
    hipLaunchKernelGGL((gdn2_attn_prologue_kernel<D, IL, false>), grid, dim3(256), 0,
                       (hipStream_t)a.stream, a, kv_groups, g.per_seq);
  return hipGetLastError();
}

}  // namespace

int norm_rope_bwd_groups(long tokens) {
  const long g = (tokens + 3) / 4;
  return (int)(g < kBwdGroups ? g : kBwdGroups);
}

size_t norm_rope_bwd_partial_bytes(long tokens, int Hq, int Hk, int d) {
  const int CH = d == 64 ? heads_per_wave<64>() : heads_per_wave<128>();
  const int chunks = (Hq + CH - 1) / CH + (Hk + CH - 1) / CH;
  return (size_t)norm_rope_bwd_groups(tokens) * chunks * d * sizeof(float);
}

#define GDN2_ROWS(FN, T)                                                         \
  (a.d == 64 ? (a.interleaved ? FN<T, 64, true>(a) : FN<T, 64, false>(a))        \
             : (a.interleaved ? FN<T, 128, true>(a) : FN<T, 128, false>(a)))

hipError_t launch_norm_rope(const NormRopeArgs& a) {
  return a.dtype == 0 ? GDN2_ROWS(run_norm_rope, bf16) : GDN2_ROWS(run_norm_rope, float);
}

hipError_t launch_norm_rope_bwd(const NormRopeArgs& a) {
  return a.dtype == 0 ? GDN2_ROWS(run_norm_rope_bwd, bf16) : GDN2_ROWS(run_norm_rope_bwd, float);
}

#undef GDN2_ROWS

long attn_prologue_groups(const AttnPrologueArgs& a) {
  const PrologueGrid g = prologue_grid(a);
  return g.units * a.Hk + g.q_groups;
}

hipError_t launch_attn_prologue(const AttnPrologueArgs& a) {
  if (a.d == 64) return a.interleaved ? run_prologue<64, true>(a) : run_prologue<64, false>(a);
  return a.interleaved ? run_prologue<128, true>(a) : run_prologue<128, false>(a);
}

}  // namespace gdn2
