// The diagonal gated recurrence on gfx950: a state per channel that decays and is written,
//     h_t = alpha_t h_{t-1} + z_t,   alpha = exp(g),  z = w v,   o_t = h_t,
// and its gradients. With e_t the gradient that reaches h_t from behind token t,
//     d_t = do_t + e_t,   e_{t-1} = alpha_t d_t,   dv = d w,  dw = d v,  dg = d alpha h_{t-1}.
//
// Both directions are scans of affine maps x -> A x + B, which compose: (A2, B2) after (A1, B1) is
// (A2 A1, A2 B1 + B2). The kernels are bound by HBM (4 flops an element forward, 8 bytes in bf16),
// so each input is read once and a sequence's state stays on the chip: one workgroup owns 64
// channels of a sequence (a row of them is one 128-byte line in bf16) and walks it in tiles of
// 32 runs of R tokens. A lane holds one run of 8 channels; the runs' maps are scanned across a
// wave's 8 runs by register exchanges and across the 4 waves through LDS, one barrier a tile,
// while the next tile's loads are in flight. A run's outputs are then the recurrence itself, from
// the state that enters it.
//
// Precision: fp32. A run's decay is exp of the sum of its logarithms, so that a state that lives
// for thousands of tokens takes one rounding of its decay per run and not per token.

#include "gdn2_attn_device.h"
#include "gdn2_stack_launch.h"

namespace gdn2 {

namespace {

constexpr int kStrip = 64;   // channels of a workgroup
constexpr int kRuns = 32;    // runs of a tile: 4 waves x 8

template <typename T> constexpr int run_tokens() { return sizeof(T) == 2 ? 4 : 2; }

// One piece of one sequence: all of it, or one of the segments that a long one is cut into.
struct Piece {
  int n;           // sequence
  long first;      // its first row
  int len;         // its tokens
  long slot;       // its first kept state
  int index;       // which segment (0 .. ), and in all the sequence's
  int begin, end;  // its tokens
};
// Unit u: segment u % per_sequence of sequence u / per_sequence; packed, sequence n's units begin at
// cu_seqlens[n] / seg + n. A unit past its sequence's end has begin > end (begin = end = 0 stands for
// a sequence without tokens).
__device__ __forceinline__ Piece piece_of(const RecurrenceArgs& a, int u) {
  Piece p;
  if (a.cu_seqlens == nullptr) {
    p.n = u / a.cut.per_sequence;
    p.index = u % a.cut.per_sequence;
    p.first = (long)p.n * a.T;
    p.len = a.T;
    p.slot = (long)p.n * ((a.T + kStateTokens - 1) / kStateTokens);
  } else {
    p.n = u;
    p.index = 0;
    if (a.cut.cut) {
      auto unit = [&](int i) { return (long)(clamped_offset(a.cu_seqlens, i, a.T) / a.cut.seg + i); };
      p.n = wave_search(a.N, u, unit);
      p.index = __builtin_amdgcn_readfirstlane(u - (int)unit(p.n));
      if (p.index < 0) p.index = 0;
    }
    const int b = uniform(clamped_offset(a.cu_seqlens, p.n, a.T)), e = uniform(clamped_offset(a.cu_seqlens, p.n + 1, a.T));
    p.first = b;
    p.len = e > b ? e - b : 0;
    p.slot = b / kStateTokens + p.n;
  }
  const long begin = (long)p.index * a.cut.seg;
  p.begin = begin < p.len || p.index == 0 ? (int)begin : p.len + 1;
  p.end = begin + a.cut.seg < p.len ? (int)begin + a.cut.seg : p.len;
  return p;
}

template <typename T>
__device__ __forceinline__ void store8_stream(T* p, const float* f) {
  if constexpr (sizeof(T) == 2) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<bf16>(f[i]);
    __builtin_nontemporal_store(v, reinterpret_cast<bf16x8*>(p));
  } else {
    __builtin_nontemporal_store(f4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f4*>(p));
    __builtin_nontemporal_store(f4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f4*>(p) + 1);
  }
}
__device__ __forceinline__ void load8f(const float* p, float* f) {
  const f4 x = reinterpret_cast<const f4*>(p)[0], y = reinterpret_cast<const f4*>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) { f[i] = x[i]; f[4 + i] = y[i]; }
}

// x of the lower and of the upper half of every group of 2 STEP lanes, in all of its lanes at the
// same place (STEP 8: the halves of a 16-lane row).
template <int STEP>
__device__ __forceinline__ void halves(float x, bool upper, float& lo, float& hi) {
  if constexpr (STEP == 8) {
    const float other = dpp_f<0x128>(x);  // row_ror:8
    lo = upper ? other : x;
    hi = upper ? x : other;
  } else if constexpr (STEP == 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(s[0]);
    hi = __uint_as_float(s[1]);
  } else {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    lo = __uint_as_float(s[0]);
    hi = __uint_as_float(s[1]);
  }
}

// One level of the scan over a wave's runs. A, H: the map of this lane's group so far, after the call
// of the group twice as large. XA, XH: the map of the runs of the group before this lane's.
template <int STEP>
__device__ __forceinline__ void scan_level(int lane, float* A, float* H, float* XA, float* XH) {
  const bool upper = (lane & STEP) != 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float al, ah, hl, hh;
    halves<STEP>(A[c], upper, al, ah);
    halves<STEP>(H[c], upper, hl, hh);
    XH[c] = fmaf(XA[c], upper ? hl : 0.f, XH[c]);
    XA[c] *= upper ? al : 1.f;
    A[c] = al * ah;
    H[c] = fmaf(ah, hl, hh);
  }
}
// The same with the backward maps L, whose later runs come first: XB, XL of the runs behind.
template <int STEP>
__device__ __forceinline__ void scan_level_both(int lane, float* A, float* H, float* L, float* XA,
                                                float* XH, float* XB, float* XL) {
  const bool upper = (lane & STEP) != 0;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float al, ah, hl, hh, ll, lh;
    halves<STEP>(A[c], upper, al, ah);
    halves<STEP>(H[c], upper, hl, hh);
    halves<STEP>(L[c], upper, ll, lh);
    XH[c] = fmaf(XA[c], upper ? hl : 0.f, XH[c]);
    XA[c] *= upper ? al : 1.f;
    XL[c] = fmaf(XB[c], upper ? 0.f : lh, XL[c]);
    XB[c] *= upper ? 1.f : ah;
    A[c] = al * ah;
    H[c] = fmaf(ah, hl, hh);
    L[c] = fmaf(al, lh, ll);
  }
}

// x through the maps of segments [s0, s1) of a sequence whose units begin at `unit`, in every lane of
// x's channels: the 32 runs take some segments each, in the order of time (BACK: against it).
// s_map: [A, H][wave][channel].
template <bool BACK>
__device__ __forceinline__ void fold_segments(const RecurrenceArgs& a, int unit, int s0, int s1, int chl, int lane,
                                              int run, float* s_map, float* x) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), cg = lane & 7;
  const int each = (s1 - s0 + kRuns - 1) / kRuns;
  float A[8], H[8], XA[8], XH[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) A[c] = XA[c] = 1.f, H[c] = XH[c] = 0.f;
  for (int i = 0; i < each; ++i) {
    const int k = run * each + i;
    if (k >= s1 - s0) break;
    const float* m = a.cut.maps + (long)(unit + (BACK ? s1 - 1 - k : s0 + k)) * 2 * a.D + chl;
    float ma[8], mh[8];
    load8f(m, ma);
    load8f(m + a.D, mh);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      A[c] *= ma[c];
      H[c] = fmaf(ma[c], H[c], mh[c]);
    }
  }
  scan_level<8>(lane, A, H, XA, XH);
  scan_level<16>(lane, A, H, XA, XH);
  scan_level<32>(lane, A, H, XA, XH);
  if (lane < 8) {
    store8(s_map + wave * kStrip + cg * 8, A);
    store8(s_map + (4 + wave) * kStrip + cg * 8, H);
  }
  lds_barrier();
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float wa[8], wh[8];
    load8f(s_map + u * kStrip + cg * 8, wa);
    load8f(s_map + (4 + u) * kStrip + cg * 8, wh);
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = fmaf(wa[c], x[c], wh[c]);
  }
}

// A tile's inputs as loaded: R tokens of 8 channels.
template <typename T, int R, int ARRAYS>
struct Raw {
  Vec8<T> x[ARRAYS][R];
};

}  // namespace

// One workgroup a (unit, 64 channels).
template <typename T, bool GATE>
__global__ void __launch_bounds__(256) gdn2_recurrence_kernel(RecurrenceArgs a, int unit0) {
  constexpr int R = run_tokens<T>(), TILE = kRuns * R, NA = GATE ? 3 : 2;
  __shared__ __attribute__((aligned(16))) float s_map[2][2][4][kStrip];  // [parity][A, H][wave][channel]
  const int strips = (a.D + kStrip - 1) / kStrip;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = unit0 + blockIdx.x / strips;
  const Piece p = piece_of(a, unit);
  if (p.begin > p.end) return;
  const int cg = lane & 7, run = wave * 8 + (lane >> 3);
  const int ch = (blockIdx.x % strips) * kStrip + cg * 8;
  const bool live = ch < a.D;
  const int chl = live ? ch : a.D - 8;  // lanes past the channels load some of the last ones
  const T* src[3] = {(const T*)a.v + chl, (const T*)a.g + chl, GATE ? (const T*)a.w + chl : nullptr};
  const long stride[3] = {a.v_stride, a.g_stride, a.w_stride};

  auto load = [&](Raw<T, R, NA>& r, int t0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      int t = t0 + run * R + i;
      t = t < p.end ? t : p.end - 1;
#pragma unroll
      for (int k = 0; k < NA; ++k) r.x[k][i].load(src[k] + (p.first + t) * stride[k]);
    }
  };
  Raw<T, R, NA> cur, next;
  if (p.begin < p.end) load(cur, p.begin);
  // The state before the tile, in every lane of its channels. The initial one goes through LDS from
  // the lanes that write the final one, which may be the same memory.
  float h[8] = {};
  if (a.s0 != nullptr) {
    if (threadIdx.x < 8) {
      load8f(a.s0 + (long)p.n * a.D + chl, h);
      store8(&s_map[1][0][0][cg * 8], h);
    }
    lds_barrier();
    load8f(&s_map[1][0][0][cg * 8], h);
  }
  int parity = 0;
  if (p.index > 0) {  // the maps of the segments before this one
    fold_segments<false>(a, unit - p.index, 0, p.index, chl, lane, run, &s_map[0][0][0][0], h);
    parity = 1;
  }
  for (int t0 = p.begin; t0 < p.end; t0 += TILE) {
    if (t0 + TILE < p.end) load(next, t0 + TILE);
    const int mine = p.end - (t0 + run * R);  // tokens of this run, from R down to none
    float al[R][8], z[R][8], A[8], H[8], XA[8], XH[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = H[c] = XH[c] = 0.f, XA[c] = 1.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float w[8], g[8];
      cur.x[0][i].to_float(z[i]);
      cur.x[1][i].to_float(g);
      if constexpr (GATE) cur.x[2][i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (GATE) z[i][c] *= w[c];
        g[c] *= kLog2e;
        if (i >= mine) g[c] = z[i][c] = 0.f;
        al[i][c] = fast_exp2(g[c]);
        A[c] += g[c];
        H[c] = fmaf(al[i][c], H[c], z[i][c]);
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = fast_exp2(A[c]);
    scan_level<8>(lane, A, H, XA, XH);
    scan_level<16>(lane, A, H, XA, XH);
    scan_level<32>(lane, A, H, XA, XH);
    if (lane < 8) {
      store8(&s_map[parity][0][wave][cg * 8], A);
      store8(&s_map[parity][1][wave][cg * 8], H);
    }
    lds_barrier();
    float x[8];  // the state before this wave's runs, then before this lane's
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float wa[8], wh[8];
      load8f(&s_map[parity][0][u][cg * 8], wa);
      load8f(&s_map[parity][1][u][cg * 8], wh);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (u == wave) x[c] = h[c];
        h[c] = fmaf(wa[c], h[c], wh[c]);
      }
    }
    parity ^= 1;
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = fmaf(XA[c], x[c], XH[c]);
    const int t = t0 + run * R;
    if (a.states != nullptr && live && mine > 0 && t % kStateTokens == 0)
      store8(a.states + (p.slot + t / kStateTokens) * a.D + ch, x);
    if (a.o != nullptr) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = fmaf(al[i][c], x[c], z[i][c]);
        if (live && i < mine) store8_stream((T*)a.o + (p.first + t + i) * a.D + ch, x);
      }
    }
    cur = next;
  }
  if (a.sN != nullptr && p.end == p.len && live && threadIdx.x < 8) store8(a.sN + (long)p.n * a.D + ch, h);
}

// The maps of the segments of long sequences, which run in parallel where sequences and channels
// are too few to fill the card: forward h -> A h + H of every segment that another follows, backward
// e -> A e + L of every segment behind another. A lane walks seg / 32 consecutive tokens of 8
// channels; the 32 runs are joined through LDS.
template <typename T, bool GATE, bool BACK>
__global__ void __launch_bounds__(256) gdn2_recurrence_maps_kernel(RecurrenceArgs a, const T* d_o, int unit0) {
  constexpr int AHEAD = 4, NA = !BACK && GATE ? 3 : 2;
  __shared__ __attribute__((aligned(16))) float s_map[2][kRuns][kStrip];
  const int strips = (a.D + kStrip - 1) / kStrip;
  const int unit = unit0 + blockIdx.x / strips;
  const Piece p = piece_of(a, unit);
  if (p.begin >= p.end || (BACK ? p.begin == 0 : p.end == p.len)) return;
  const int cg = threadIdx.x & 7, run = threadIdx.x >> 3;
  const int ch = (blockIdx.x % strips) * kStrip + cg * 8;
  const int chl = ch < a.D ? ch : a.D - 8;
  const T* src[3] = {(const T*)a.g + chl, BACK ? d_o + chl : (const T*)a.v + chl, GATE ? (const T*)a.w + chl : nullptr};
  const long stride[3] = {a.g_stride, BACK ? (long)a.D : a.v_stride, a.w_stride};
  const int each = a.cut.seg / kRuns;
  // tokens t0, t0 + 1, .. (BACK: t0, t0 - 1, ..), those past the end counting as none
  const int t0 = p.begin + run * each + (BACK ? each - 1 : 0);
  float G[8], H[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) G[c] = H[c] = 0.f;
  auto load = [&](Raw<T, AHEAD, NA>& r, int i0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      int t = BACK ? t0 - i0 - i : t0 + i0 + i;
      t = t < p.end ? t : p.end - 1;
      t = t > 0 ? t : 0;
#pragma unroll
      for (int k = 0; k < NA; ++k) r.x[k][i].load(src[k] + (p.first + t) * stride[k]);
    }
  };
  Raw<T, AHEAD, NA> cur, next;
  load(cur, 0);
  for (int i0 = 0; i0 < each; i0 += AHEAD) {
    if (i0 + AHEAD < each) load(next, i0 + AHEAD);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool in = i0 + i < each && (BACK ? t0 - i0 - i : t0 + i0 + i) < p.end;
      float g[8], x[8], w[8];
      cur.x[0][i].to_float(g);
      cur.x[1][i].to_float(x);
      if constexpr (NA == 3) cur.x[2][i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (NA == 3) x[c] *= w[c];
        g[c] *= kLog2e;
        if (!in) g[c] = x[c] = 0.f;
        const float al = fast_exp2(g[c]);
        G[c] += g[c];
        H[c] = BACK ? al * (x[c] + H[c]) : fmaf(al, H[c], x[c]);
      }
    }
    cur = next;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) G[c] = fast_exp2(G[c]);
  store8(&s_map[0][run][cg * 8], G);
  store8(&s_map[1][run][cg * 8], H);
  lds_barrier();
  if (threadIdx.x < kStrip) {
    const int c = (blockIdx.x % strips) * kStrip + threadIdx.x;
    float A = 1.f, B = 0.f;
#pragma unroll 8
    for (int k = 0; k < kRuns; ++k) {
      const int r = BACK ? kRuns - 1 - k : k;
      A *= s_map[0][r][threadIdx.x];
      B = fmaf(s_map[0][r][threadIdx.x], B, s_map[1][r][threadIdx.x]);
    }
    if (c < a.D) {
      a.cut.maps[(long)unit * 2 * a.D + c] = A;
      a.cut.maps[((long)unit * 2 + 1) * a.D + c] = B;
    }
  }
}

// Gradients, tiles from the last to the first: the states come from the kept ones, the carry e runs
// against time. One more workgroup row behind the sequences (packed batches) writes zeros to the
// gradients of rows that belong to none.
template <typename T, bool GATE>
__global__ void __launch_bounds__(256) gdn2_recurrence_bwd_kernel(RecurrenceBwdArgs b, int unit0) {
  constexpr int R = 2, TILE = kRuns * R, NA = GATE ? 4 : 3;
  static_assert(TILE == kStateTokens, "a tile starts at a kept state");
  __shared__ __attribute__((aligned(16))) float s_map[2][3][4][kStrip];  // [parity][A, H, L][wave][channel]
  const RecurrenceArgs& a = b.f;
  const int strips = (a.D + kStrip - 1) / kStrip;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int unit = unit0 + blockIdx.x / strips;
  const int cg = lane & 7, run = wave * 8 + (lane >> 3);
  const int ch = (blockIdx.x % strips) * kStrip + cg * 8;
  const bool live = ch < a.D;
  const int chl = live ? ch : a.D - 8;
  if (unit == a.cut.units) {
    const int first = clamped_offset(a.cu_seqlens, 0, a.T), last = clamped_offset(a.cu_seqlens, a.N, a.T);
    const float zero[8] = {};
    for (int t = run; t < a.T; t += kRuns)
      if (live && (t < first || t >= last)) {
        store8((T*)b.dv + (long)t * a.D + ch, zero);
        store8((T*)b.dg + (long)t * a.D + ch, zero);
        if (GATE) store8((T*)b.dw + (long)t * a.D + ch, zero);
      }
    return;
  }
  const Piece p = piece_of(a, unit);
  if (p.begin > p.end) return;
  const T* src[4] = {(const T*)a.v + chl, (const T*)a.g + chl, (const T*)b.d_o + chl, GATE ? (const T*)a.w + chl : nullptr};
  const long stride[4] = {a.v_stride, a.g_stride, (long)a.D, a.w_stride};

  float e[8];  // the gradient of the state behind the tile, in every lane of its channels
#pragma unroll
  for (int c = 0; c < 8; ++c) e[c] = 0.f;
  if (b.d_sN != nullptr) load8f(b.d_sN + (long)p.n * a.D + chl, e);
  int parity = 0;

  auto load = [&](Raw<T, R, NA>& r, float* h, int t0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      int t = t0 + run * R + i;
      t = t < p.end ? t : p.end - 1;
#pragma unroll
      for (int k = 0; k < NA; ++k) r.x[k][i].load(src[k] + (p.first + t) * stride[k]);
    }
    load8f(a.states + (p.slot + t0 / kStateTokens) * a.D + chl, h);
  };
  Raw<T, R, NA> cur, next;
  float h[8], hnext[8];
  const int t_last = p.begin + (p.end - 1 - p.begin) / TILE * TILE;
  if (p.begin < p.end) load(cur, h, t_last);
  if (p.end < p.len) {  // the maps of the segments behind this one
    const int count = (p.len + a.cut.seg - 1) / a.cut.seg;
    fold_segments<true>(a, unit - p.index, p.index + 1, count, chl, lane, run, &s_map[0][0][0][0], e);
    parity = 1;
  }
  for (int t0 = t_last; p.begin < p.end && t0 >= p.begin; t0 -= TILE) {
    if (t0 > p.begin) load(next, hnext, t0 - TILE);
    const int mine = p.end - (t0 + run * R);
    float al[R][8], z[R][8], d[R][8], A[8], H[8], L[8], XA[8], XH[8], XB[8], XL[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = H[c] = L[c] = XH[c] = XL[c] = 0.f, XA[c] = XB[c] = 1.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float w[8], g[8];
      cur.x[0][i].to_float(z[i]);
      cur.x[1][i].to_float(g);
      cur.x[2][i].to_float(d[i]);
      if constexpr (GATE) cur.x[3][i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (GATE) z[i][c] *= w[c];
        g[c] *= kLog2e;
        if (i >= mine) g[c] = z[i][c] = d[i][c] = 0.f;
        al[i][c] = fast_exp2(g[c]);
        A[c] += g[c];
        H[c] = fmaf(al[i][c], H[c], z[i][c]);
      }
    }
#pragma unroll
    for (int i = R - 1; i >= 0; --i)
#pragma unroll
      for (int c = 0; c < 8; ++c) L[c] = al[i][c] * (d[i][c] + L[c]);
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = fast_exp2(A[c]);
    scan_level_both<8>(lane, A, H, L, XA, XH, XB, XL);
    scan_level_both<16>(lane, A, H, L, XA, XH, XB, XL);
    scan_level_both<32>(lane, A, H, L, XA, XH, XB, XL);
    if (lane < 8) {
      store8(&s_map[parity][0][wave][cg * 8], A);
      store8(&s_map[parity][1][wave][cg * 8], H);
      store8(&s_map[parity][2][wave][cg * 8], L);
    }
    lds_barrier();
    float x[8], y[8];  // the state before this lane's run, the gradient behind it
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float wa[8], wh[8], ba[8], bl[8];
      load8f(&s_map[parity][0][u][cg * 8], wa);
      load8f(&s_map[parity][1][u][cg * 8], wh);
      load8f(&s_map[parity][0][3 - u][cg * 8], ba);
      load8f(&s_map[parity][2][3 - u][cg * 8], bl);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if (u == wave) x[c] = h[c];
        h[c] = fmaf(wa[c], h[c], wh[c]);
        if (3 - u == wave) y[c] = e[c];
        e[c] = fmaf(ba[c], e[c], bl[c]);
      }
    }
    parity ^= 1;
    float before[R][8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      x[c] = fmaf(XA[c], x[c], XH[c]);
      y[c] = fmaf(XB[c], y[c], XL[c]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        before[i][c] = x[c];
        x[c] = fmaf(al[i][c], x[c], z[i][c]);
      }
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      float v[8], w[8], gv[8], gg[8], gw[8];
      cur.x[0][i].to_float(v);
      if constexpr (GATE) cur.x[3][i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float dt = d[i][c] + y[c];
        y[c] = al[i][c] * dt;
        gv[c] = GATE ? dt * w[c] : dt;
        gw[c] = dt * v[c];
        gg[c] = y[c] * before[i][c];
      }
      if (live && i < mine) {
        const long at = (p.first + t0 + run * R + i) * a.D + ch;
        store8_stream((T*)b.dv + at, gv);
        store8_stream((T*)b.dg + at, gg);
        if constexpr (GATE) store8_stream((T*)b.dw + at, gw);
      }
    }
    cur = next;
#pragma unroll
    for (int c = 0; c < 8; ++c) h[c] = hnext[c];
  }
  if (b.d_s0 != nullptr && p.begin == 0 && live && threadIdx.x < 8) store8(b.d_s0 + (long)p.n * a.D + ch, e);
}

// L tokens of every sequence against a pool of states: a lane takes 8 channels of one sequence, its
// state in registers. Bytes are few; the call is bound by its latency, so the inputs of up to 4
// tokens are loaded at once.
template <typename T, bool GATE>
__global__ void __launch_bounds__(64) gdn2_recurrence_tokens_kernel(RecurrenceTokensArgs a) {
  constexpr int AHEAD = 4, NA = GATE ? 3 : 2;
  const int groups = a.D / 8;
  const long id = (long)blockIdx.x * 64 + threadIdx.x;
  const int n = (int)(id / groups);
  if (n >= a.N) return;
  const int ch = (int)(id % groups) * 8;
  const int slot = a.indices != nullptr ? a.indices[n] : n;
  if (slot < 0 || slot >= a.P) return;
  const int keep = a.commit != nullptr ? a.commit[n] : a.L;
  float* const state = a.pool + (long)slot * a.D + ch;
  const T* src[3] = {(const T*)a.v + ch, (const T*)a.g + ch, GATE ? (const T*)a.w + ch : nullptr};
  const long stride[3] = {a.v_stride, a.g_stride, a.w_stride};
  float h[8];
  load8f(state, h);
  for (int t0 = 0; t0 < a.L; t0 += AHEAD) {
    Raw<T, AHEAD, NA> r;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const long t = (long)n * a.L + (t0 + i < a.L ? t0 + i : a.L - 1);
#pragma unroll
      for (int k = 0; k < NA; ++k) r.x[k][i].load(src[k] + t * stride[k]);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int t = t0 + i;
      if (t >= a.L) break;
      float z[8], g[8], w[8];
      r.x[0][i].to_float(z);
      r.x[1][i].to_float(g);
      if constexpr (GATE) r.x[2][i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        if constexpr (GATE) z[c] *= w[c];
        h[c] = fmaf(fast_exp2(g[c] * kLog2e), h[c], z[c]);
      }
      store8((T*)a.o + ((long)n * a.L + t) * a.D + ch, h);
      if (a.step_states != nullptr) store8(a.step_states + ((long)n * a.L + t) * a.D + ch, h);
      if (t + 1 == keep || (t + 1 == a.L && keep > a.L)) store8(state, h);
    }
  }
}

long recurrence_state_slots(bool packed, int B, int T, int N) {
  return packed ? (long)T / kStateTokens + N : (long)B * ((T + kStateTokens - 1) / kStateTokens);
}

static int strips_of(int D) { return (D + kStrip - 1) / kStrip; }

RecurrenceCut recurrence_cut(bool packed, int B, int T, int D, int N) {
  constexpr int TILE = 128;
  RecurrenceCut c{};
  const long strips = strips_of(D), tokens = (long)B * T;
  c.cut = false;
  c.seg = T > 0 ? T : 1;
  c.per_sequence = 1;
  c.units = N;
  if (T < 6 * TILE || N == 0) return c;
  // tokens of a unit where everything is cut into 512 of (unit, strip), two for a compute unit
  long seg = ((tokens * strips + 511) / 512 + TILE - 1) / TILE * TILE;
  if (seg < 2 * TILE) seg = 2 * TILE;
  if (N * strips > 96) {
    if (!packed) return c;
    seg *= 2;
  }
  if (seg >= T) return c;
  c.cut = true;
  c.seg = (int)seg;
  c.per_sequence = packed ? 1 : (int)((T + seg - 1) / seg);
  c.units = packed ? (int)(T / seg + N) : N * c.per_sequence;
  return c;
}
long recurrence_groups(const RecurrenceCut& c, int D) { return ((long)c.units + 1) * strips_of(D); }
size_t recurrence_workspace_bytes(const RecurrenceCut& c, int D) {
  return c.cut ? (size_t)c.units * 2 * D * sizeof(float) : 0;
}

namespace {

template <typename T, bool GATE>
hipError_t forward(const RecurrenceArgs& a) {
  const unsigned strips = (unsigned)strips_of(a.D);
  const hipStream_t st = (hipStream_t)a.stream;
  const dim3 grid((unsigned)a.cut.units * strips), block(256);
  if (a.cut.cut) hipLaunchKernelGGL((gdn2_recurrence_maps_kernel<T, GATE, false>), grid, block, 0, st, a, (const T*)nullptr, 0);
  hipLaunchKernelGGL((gdn2_recurrence_kernel<T, GATE>), grid, block, 0, st, a, 0);
  return hipGetLastError();
}

template <typename T, bool GATE>
hipError_t backward(const RecurrenceBwdArgs& b) {
  const RecurrenceArgs& a = b.f;
  const unsigned strips = (unsigned)strips_of(a.D);
  const hipStream_t st = (hipStream_t)a.stream;
  const unsigned units = (unsigned)a.cut.units;
  if (a.cut.cut) hipLaunchKernelGGL((gdn2_recurrence_maps_kernel<T, false, true>), dim3(units * strips), dim3(256), 0, st, a, (const T*)b.d_o, 0);
  hipLaunchKernelGGL((gdn2_recurrence_bwd_kernel<T, GATE>), dim3((units + (a.cu_seqlens != nullptr)) * strips), dim3(256), 0, st, b, 0);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_recurrence(const RecurrenceArgs& a) {
  if (a.dtype == 0) return a.w ? forward<bf16, true>(a) : forward<bf16, false>(a);
  return a.w ? forward<float, true>(a) : forward<float, false>(a);
}

hipError_t launch_recurrence_bwd(const RecurrenceBwdArgs& b) {
  if (b.f.dtype == 0) return b.f.w ? backward<bf16, true>(b) : backward<bf16, false>(b);
  return b.f.w ? backward<float, true>(b) : backward<float, false>(b);
}

hipError_t launch_recurrence_tokens(const RecurrenceTokensArgs& a) {
  const dim3 grid((unsigned)(((long)a.N * (a.D / 8) + 63) / 64)), block(64);
  const hipStream_t st = (hipStream_t)a.stream;
  if (a.dtype == 0) {
    if (a.w) hipLaunchKernelGGL((gdn2_recurrence_tokens_kernel<bf16, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((gdn2_recurrence_tokens_kernel<bf16, false>), grid, block, 0, st, a);
  } else {
    if (a.w) hipLaunchKernelGGL((gdn2_recurrence_tokens_kernel<float, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((gdn2_recurrence_tokens_kernel<float, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace gdn2
