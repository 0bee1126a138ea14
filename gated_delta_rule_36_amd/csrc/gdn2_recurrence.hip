// The diagonal gated recurrence on gfx950: a state per channel that decays and is written,
//     h_t = alpha_t h_{t-1} + z_t,   alpha = exp(g),  z = w v,   o_t = h_t,
// and its gradients. With e_t the gradient that reaches h_t from behind token t,
//     d_t = do_t + e_t,   e_{t-1} = alpha_t d_t,   dv = d w,  dw = d v,  dg = d alpha h_{t-1}.
//
// Both directions are scans of affine maps x -> A x + B, which compose: (A2, B2) after (A1, B1) is
// (A2 A1, A2 B1 + B2). The kernels are bound by HBM (4 flops an element forward, 8 bytes in bf16),
// so each input is read once and a sequence's state stays on the chip: one workgroup owns 64
// channels of a sequence (a row of them is one 128-byte line in bf16) and walks it in tiles of
// 32 or 64 runs of R tokens. A lane holds one run of 8 channels; the runs' maps are scanned across a
// wave's 8 runs by register exchanges and across the 4 or 8 waves through LDS, one barrier a tile,
// while the next tile's loads are in flight. A run's outputs are then the recurrence itself, from
// the state that enters it. 8 x 2048 tokens of 2048 channels in bf16: 58 us forward (4.6 TB/s), 103
// backward (4.6), where a copy moves 5.4 TB/s and inputs at a stride of 4224 bytes run 50 forward.
// Long sequences of few channels are cut into segments (see below), whose inputs are read again.
//
// Precision: fp32. A run's decay is exp of the sum of its logarithms, so that a state that lives
// for thousands of tokens takes one rounding of its decay per run and not per token.

#include "gdn2_attn_device.h"
#include "gdn2_stack_device.h"
#include "gdn2_stack_launch.h"

namespace gdn2 {

namespace {

constexpr int kStrip = 64;   // channels of a workgroup
constexpr int kRuns = 32;    // runs of 4 waves (of the maps' pass)

__host__ __device__ constexpr int strips_of(int D) { return (D + kStrip - 1) / kStrip; }

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
// Unit u: segment u % per_sequence of sequence u / per_sequence; packed and cut, sequence n's units
// begin at cu_seqlens[n] / seg + n. A unit that no segment has (in front of the first sequence's, past
// a sequence's end) has begin > end; a sequence without tokens has begin = end = 0.
__device__ __forceinline__ Piece piece_of(const RecurrenceArgs& a, int u) {
  Piece p;
  bool none = false;
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
      p.index = uniform(u - (int)unit(p.n));
      none = p.index < 0;
      if (none) p.index = 0;
    }
    const int b = uniform(clamped_offset(a.cu_seqlens, p.n, a.T)), e = uniform(clamped_offset(a.cu_seqlens, p.n + 1, a.T));
    p.first = b;
    p.len = e > b ? e - b : 0;
    p.slot = b / kStateTokens + p.n;
  }
  const long begin = (long)p.index * a.cut.seg;
  none = none || (p.index > 0 && begin >= p.len);
  p.begin = none ? p.len + 1 : (int)begin;
  p.end = begin + a.cut.seg < p.len ? (int)begin + a.cut.seg : p.len;
  return p;
}

// What a launch knows of its rows. Lines of 128 bytes that two strips share stay in the caches, for
// both loads and stores; outputs in whole lines go past them; inputs too where they are too many to
// be there (see streamed()).
enum { kSharedLines = 0, kLines = 1, kStream = 2 };

// The 8 channels of a lane in its strip: 4 from `lo` on and 4 from `hi` on, so that 8 lanes' accesses of
// 16 bytes make one line: 8 in a row in bf16, in fp32 4 of each half of the strip. `own`: of the 64
// channels in the order of the lanes (8 cg + c), the place in the strip.
template <typename T>
struct Channels {
  int lo, hi;           // places in the strip
  bool in_lo, in_hi;    // inside the D channels
  int load_lo, load_hi; // lanes past the channels load some of the last ones
  __device__ __forceinline__ Channels(int cg, int strip, int D) {
    lo = sizeof(T) == 2 ? cg * 8 : cg * 4;
    hi = sizeof(T) == 2 ? cg * 8 + 4 : 32 + cg * 4;
    in_lo = strip + lo < D;
    in_hi = strip + hi < D;
    load_lo = in_lo ? lo : D - (sizeof(T) == 2 ? 8 : 4) - strip;
    load_hi = in_hi ? hi : D - 4 - strip;
  }
  static __device__ __forceinline__ int place(int own) {
    return sizeof(T) == 2 ? own : (own >> 3) * 4 + (own & 3) + (own & 4) * 8;
  }
  template <int MODE>
  __device__ __forceinline__ void load(Vec8<T>& r, const T* p) const {  // p: the strip in a row
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    const u4* a = reinterpret_cast<const u4*>(p + load_lo);
    if constexpr (sizeof(T) == 2) {
      r.r = __builtin_bit_cast(uint4, MODE == kStream ? __builtin_nontemporal_load(a) : *a);
    } else {
      const u4* b = reinterpret_cast<const u4*>(p + load_hi);
      r.r0 = __builtin_bit_cast(uint4, MODE == kStream ? __builtin_nontemporal_load(a) : *a);
      r.r1 = __builtin_bit_cast(uint4, MODE == kStream ? __builtin_nontemporal_load(b) : *b);
    }
  }
  template <int MODE>
  __device__ __forceinline__ void store(T* p, const float* f) const {
    if constexpr (MODE == kSharedLines && sizeof(T) == 2) {
      if (in_lo) store8(p + lo, f);
    } else if constexpr (MODE == kSharedLines) {
      store_f(p, f);
    } else if constexpr (sizeof(T) == 2) {
      if (in_lo) store8_stream(p + lo, f);
    } else {
      if (in_lo) __builtin_nontemporal_store(f4{f[0], f[1], f[2], f[3]}, reinterpret_cast<f4*>(p + lo));
      if (in_hi) __builtin_nontemporal_store(f4{f[4], f[5], f[6], f[7]}, reinterpret_cast<f4*>(p + hi));
    }
  }
  // the same channels of an array in fp32
  __device__ __forceinline__ void load_f(const float* p, float* f) const {
    const int second = sizeof(T) == 2 ? load_lo + 4 : load_hi;
    const f4 x = *reinterpret_cast<const f4*>(p + load_lo), y = *reinterpret_cast<const f4*>(p + second);
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = x[i]; f[4 + i] = y[i]; }
  }
  __device__ __forceinline__ void store_f(float* p, const float* f) const {
    if (in_lo) *reinterpret_cast<f4*>(p + lo) = f4{f[0], f[1], f[2], f[3]};
    if (in_hi) *reinterpret_cast<f4*>(p + hi) = f4{f[4], f[5], f[6], f[7]};
  }
};

// The workgroup's (unit, strip). Where rows do not begin at lines, neighbouring strips share lines, and
// each XCD (workgroups start on them in turn) takes a run of neighbours so that its L2 holds them once:
// the grid is rounded up to a multiple of 8, and false says that this workgroup has nothing.
__device__ __forceinline__ bool my_group(const RecurrenceArgs& a, int units, int& unit, int& strip) {
  const int strips = strips_of(a.D);
  int i = blockIdx.x;
  if (a.shared_lines) {
    const int each = gridDim.x >> 3;
    i = (blockIdx.x & 7) * each + (blockIdx.x >> 3);
    if (i >= units * strips) return false;
  }
  unit = i / strips;
  strip = i % strips * kStrip;
  return true;
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

// x, a value of the lane's own channel `c`, through the maps of segments [s0, s1) of a
// sequence whose units begin at `unit`: the runs take some segments each, in the order of time (BACK:
// against it). s_map: [A, H][wave][channel].
template <bool BACK, int NW, typename T>
__device__ __forceinline__ void fold_segments(const RecurrenceArgs& a, int unit, int s0, int s1, int strip, const Channels<T>& cn,
                                              int lane, int run, int c, float* s_map, float& x) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), cg = lane & 7;
  const int each = (s1 - s0 + NW * 8 - 1) / (NW * 8);
  float A[8], H[8], XA[8], XH[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) A[j] = XA[j] = 1.f, H[j] = XH[j] = 0.f;
  for (int i = 0; i < each; ++i) {
    const int k = run * each + i;
    if (k >= s1 - s0) break;
    const float* m = a.cut.maps + (long)(unit + (BACK ? s1 - 1 - k : s0 + k)) * 2 * a.D + strip;
    float ma[8], mh[8];
    cn.load_f(m, ma);
    cn.load_f(m + a.D, mh);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      A[j] *= ma[j];
      H[j] = fmaf(ma[j], H[j], mh[j]);
    }
  }
  scan_level<8>(lane, A, H, XA, XH);
  scan_level<16>(lane, A, H, XA, XH);
  scan_level<32>(lane, A, H, XA, XH);
  if (lane < 8) {
    store8(s_map + wave * kStrip + cg * 8, A);
    store8(s_map + (NW + wave) * kStrip + cg * 8, H);
  }
  lds_barrier();
#pragma unroll
  for (int u = 0; u < NW; ++u) x = fmaf(s_map[u * kStrip + c], x, s_map[(NW + u) * kStrip + c]);
}

// A tile's inputs as loaded: R tokens of 8 channels.
template <typename T, int R, int ARRAYS>
struct Raw {
  Vec8<T> x[ARRAYS][R];
};

}  // namespace

// Rows t0 + row of up to ARRAYS inputs: a uniform base and one 32-bit offset a lane (strides are at most
// kMaxStride, so that the rows of a tile stay within it). At an instant each array is at another of the
// run's tokens.
template <typename T, int ARRAYS>
struct Rows {
  const T* src[ARRAYS];  // uniform: the strip in the sequence's first row
  long stride[ARRAYS];
  template <int MODE, int R>
  __device__ __forceinline__ void load(Raw<T, R, ARRAYS>& r, const Channels<T>& cn, int t0, int row0, int rows) const {
#pragma unroll
    for (int j = 0; j < R; ++j) {
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
        const int i = (j + k) % R;
        const int row = row0 + i < rows ? row0 + i : rows - 1;
        cn.template load<MODE>(r.x[k][i], src[k] + t0 * stride[k] + (unsigned)__umul24(row, (int)stride[k]));
      }
    }
  }
};

// Zeros in the rows of a packed batch that belong to no sequence, 64 channels a workgroup. (One workgroup
// for all of them: at 131072 rows of which 4096 are in sequences the training forward takes 270 us and the
// backward 750, at 64 channels as at 2048.)
template <typename T>
__device__ __forceinline__ void zero_outside(const RecurrenceArgs& a, T* x, const Channels<T>& cn, int strip) {
  const int first = clamped_offset(a.cu_seqlens, 0, a.T), last = clamped_offset(a.cu_seqlens, a.N, a.T);
  const float zero[8] = {};
  for (int t = threadIdx.x >> 3; t < a.T; t += blockDim.x >> 3)
    if (t < first || t >= last) cn.template store<kSharedLines>(x + (long)t * a.D + strip, zero);
}

// How a cut forward runs. Short segments: a pass for the segments' maps h -> A h + H (below), then all
// segments at once (kWhole), each from the state that the maps before it give. Long ones (see
// recurrence_cut), which may forget what came before them: the first pass walks every segment from a zero
// state (the first segment from the initial one), leaves its map, and writes the outputs from the tile on
// in front of which the decay has taken everything of the state before (A = 0 in fp32 in all channels of
// the strip); the second pass walks the tiles before that one again, from the state that the earlier
// maps give. 32768 tokens of 2048 channels in bf16, in us (a pass for the maps and one for all outputs: 178
// whatever the decays are):
//   one token in 10 a reset to e^-5       136   (every tile of a segment but the first two is final)
//   alpha 0.92 on average                 155
//   nothing forgotten within a segment    185   (both passes read everything: 14 bytes an element)
enum { kWhole = 0, kFirst = 1, kSecond = 2 };

// One workgroup a (unit, 64 channels), and where states are kept for the backward of a packed batch one
// row of them more, for the rows of no sequence. A tile's registers are filled with the next tile's inputs as
// soon as its values are widened to fp32, so that loads are in flight during the scan and the stores.
template <typename T, bool GATE, int NW, int MODE, int PASS>
__global__ void __launch_bounds__(64 * NW) gdn2_recurrence_kernel(RecurrenceArgs a) {
  constexpr int R = run_tokens<T>(), TILE = NW * 8 * R, NA = GATE ? 3 : 2;
  __shared__ __attribute__((aligned(16))) float s_map[2][2][NW][kStrip];  // [parity][A, H][wave][channel]
  __shared__ __attribute__((aligned(16))) float s_in[NW][kStrip];         // the state before a wave's runs
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int unit, strip;
  if (!my_group(a, a.cut.units + (PASS != kSecond && a.zero_rest), unit, strip)) return;
  const int cg = lane & 7, run = wave * 8 + (lane >> 3);
  const Channels<T> cn(cg, strip, a.D);
  if (PASS != kSecond && unit == a.cut.units) {
    zero_outside(a, (T*)a.o, cn, strip);
    return;
  }
  const Piece p = piece_of(a, unit);
  if (p.begin > p.end || (PASS == kSecond && p.index == 0)) return;
  // the channel whose state this lane carries from tile to tile
  const int own = cg * 8 + (lane >> 3), owned = strip + Channels<T>::place(own), och = owned < a.D ? owned : a.D - 1;
  Rows<T, NA> in;
  in.src[0] = (const T*)a.v + p.first * a.v_stride + strip;
  in.src[1] = (const T*)a.g + p.first * a.g_stride + strip;
  in.stride[0] = a.v_stride;
  in.stride[1] = a.g_stride;
  if constexpr (GATE) {
    in.src[2] = (const T*)a.w + p.first * a.w_stride + strip;
    in.stride[2] = a.w_stride;
  }
  T* const out = a.o != nullptr ? (T*)a.o + p.first * a.D + strip : nullptr;
  float* const kept = a.states != nullptr ? a.states + p.slot * a.D + strip : nullptr;

  Raw<T, R, NA> r;
  if (p.begin < p.end) in.template load<MODE>(r, cn, p.begin, run * R, p.end - p.begin);
  int end = p.end;  // of the tiles
  // of the first pass: how much of the state before the unit is left (own channel), the tokens whose outputs still depend on it
  float reach = p.index > 0 ? 1.f : 0.f;
  int open = 0;
  float* const map = PASS != kWhole ? a.cut.maps + (long)unit * 2 * a.D + och : nullptr;
  int* const opened = PASS != kWhole ? reinterpret_cast<int*>(a.cut.maps + (long)a.cut.units * 2 * a.D) +
                                           (long)unit * strips_of(a.D) + strip / kStrip
                                     : nullptr;
  // The initial state goes through LDS from the lanes that write the final one, which may be the same
  // memory.
  float h = 0.f;
  if (PASS != kSecond && (PASS == kWhole || p.index == 0) && a.s0 != nullptr) {
    if (wave == 0) s_map[1][0][0][own] = a.s0[(long)p.n * a.D + och];
    lds_barrier();
    h = s_map[1][0][0][own];
  }
  int parity = 0;
  if (PASS != kFirst && p.index > 0) {  // the maps of the segments before this one
    const int still = PASS == kSecond ? uniform(*opened) : 0;
    fold_segments<false, NW>(a, unit - p.index, 0, p.index, strip, cn, lane, run, own, &s_map[0][0][0][0], h);
    parity = 1;
    // (a state that is not finite stays so, however far it decays)
    if (PASS == kSecond && __all(fabsf(h) < INFINITY) && still < p.end - p.begin) end = p.begin + still;
  }
  for (int t0 = p.begin; t0 < end; t0 += TILE) {
    const int mine = p.end - (t0 + run * R);  // tokens of this run, from R down to none
    float al[R][8], z[R][8], A[8], H[8], XA[8], XH[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = H[c] = XH[c] = 0.f, XA[c] = 1.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float w[8], g[8];
      r.x[0][i].to_float(z[i]);
      r.x[1][i].to_float(g);
      if constexpr (GATE) r.x[2][i].to_float(w);
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
    if (t0 + TILE < end) in.template load<MODE>(r, cn, t0 + TILE, run * R, p.end - t0 - TILE);
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
    // each lane joins the waves' maps for its own channel and hands the state before this wave's runs
    // to the lanes that hold the channel
    float xin = h;
    const bool settled = PASS != kFirst || __all(reach == 0.f);
#pragma unroll
    for (int u = 0; u < NW; ++u) {
      const float wa = s_map[parity][0][u][own];
      if (u == wave) xin = h;
      h = fmaf(wa, h, s_map[parity][1][u][own]);
      if constexpr (PASS == kFirst) reach = reach == 0.f ? 0.f : reach * wa;  // (0 stays 0, however much the decay grows)
    }
    parity ^= 1;
    if (!settled) {
      open += TILE;
      continue;
    }
    s_in[wave][own] = xin;
    float x[8];
    load8f(&s_in[wave][cg * 8], x);
#pragma unroll
    for (int c = 0; c < 8; ++c) x[c] = fmaf(XA[c], x[c], XH[c]);
    const int t = t0 + run * R;
    if (kept != nullptr && mine > 0 && t % kStateTokens == 0) cn.store_f(kept + (long)(t / kStateTokens) * a.D, x);
    if (out != nullptr) {
      T* const to = out + (long)t0 * a.D;
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = fmaf(al[i][c], x[c], z[i][c]);
        if (i < mine) cn.template store<MODE>(to + (unsigned)__umul24(run * R + i, a.D), x);
      }
    }
  }
  if (wave == 0 && owned < a.D) {
    if constexpr (PASS == kFirst) {
      map[0] = reach;
      map[a.D] = h;
      if (lane == 0) *opened = open;
    }
    // (where the second pass ended early, nothing of the state before the unit is left at its end)
    if (a.sN != nullptr && p.end == p.len && (PASS != kFirst || p.index == 0))
      a.sN[(long)p.n * a.D + och] = end < p.end ? map[a.D] : h;
  }
}

// The maps of the segments of long sequences, which run in parallel where sequences and channels
// are too few to fill the card: forward h -> A h + H of every segment that another follows, backward
// e -> A e + L of every segment behind another. A lane walks seg / 32 consecutive tokens of 8
// channels; the 32 runs are joined through LDS.
template <typename T, bool GATE, bool BACK>
__global__ void __launch_bounds__(256) gdn2_recurrence_maps_kernel(RecurrenceArgs a, const T* d_o) {
  constexpr int AHEAD = 4, NA = !BACK && GATE ? 3 : 2;
  __shared__ __attribute__((aligned(16))) float s_map[2][kRuns][kStrip];
  int unit, strip;
  if (!my_group(a, a.cut.units, unit, strip)) return;
  const Piece p = piece_of(a, unit);
  if (p.begin >= p.end || (BACK ? p.begin == 0 : p.end == p.len)) return;
  const int cg = threadIdx.x & 7, run = threadIdx.x >> 3;
  const Channels<T> cn(cg, strip, a.D);
  const T* src[3] = {(const T*)a.g + strip, (BACK ? d_o : (const T*)a.v) + strip, GATE ? (const T*)a.w + strip : nullptr};
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
      for (int k = 0; k < NA; ++k) cn.template load<kLines>(r.x[k][i], src[k] + (p.first + t) * stride[k]);
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
    const int c = strip + Channels<T>::place(threadIdx.x);
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
// against time. One more workgroup row behind the units (packed batches) writes zeros to the
// gradients of rows that belong to no sequence.
template <typename T, bool GATE, int NW, int MODE>
__global__ void __launch_bounds__(64 * NW) gdn2_recurrence_bwd_kernel(RecurrenceBwdArgs b) {
  constexpr int R = 2, TILE = NW * 8 * R, NA = GATE ? 4 : 3;
  static_assert(TILE % kStateTokens == 0, "a tile starts at a kept state");
  __shared__ __attribute__((aligned(16))) float s_map[2][3][NW][kStrip];  // [parity][A, H, L][wave][channel]
  __shared__ __attribute__((aligned(16))) float s_in[2][NW][kStrip];      // the state before a wave's runs, the gradient behind
  const RecurrenceArgs& a = b.f;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int unit, strip;
  if (!my_group(a, a.cut.units + a.zero_rest, unit, strip)) return;
  const int cg = lane & 7, run = wave * 8 + (lane >> 3);
  const Channels<T> cn(cg, strip, a.D);
  if (unit == a.cut.units) {
    zero_outside(a, (T*)b.dv, cn, strip);
    zero_outside(a, (T*)b.dg, cn, strip);
    if (GATE) zero_outside(a, (T*)b.dw, cn, strip);
    return;
  }
  const Piece p = piece_of(a, unit);
  if (p.begin > p.end) return;
  const int own = cg * 8 + (lane >> 3), owned = strip + Channels<T>::place(own), och = owned < a.D ? owned : a.D - 1;
  Rows<T, NA> in;
  in.src[0] = (const T*)a.v + p.first * a.v_stride + strip;
  in.src[1] = (const T*)a.g + p.first * a.g_stride + strip;
  in.src[2] = (const T*)b.d_o + p.first * a.D + strip;
  in.stride[0] = a.v_stride;
  in.stride[1] = a.g_stride;
  in.stride[2] = a.D;
  if constexpr (GATE) {
    in.src[3] = (const T*)a.w + p.first * a.w_stride + strip;
    in.stride[3] = a.w_stride;
  }
  const float* const kept = a.states + p.slot * a.D + och;
  const long out = p.first * a.D + strip;

  // of the lane's own channel: the gradient of the state behind the tile, the state before it
  float e = b.d_sN != nullptr ? b.d_sN[(long)p.n * a.D + och] : 0.f, hnext = 0.f;
  int parity = 0;
  Raw<T, R, NA> r;
  auto load = [&](int t0) {
    in.template load<MODE>(r, cn, t0, run * R, p.end - t0);
    hnext = kept[(long)(t0 / kStateTokens) * a.D];
  };
  const int t_last = p.begin + (p.end - 1 - p.begin) / TILE * TILE;
  if (p.begin < p.end) load(t_last);
  if (p.end < p.len) {  // the maps of the segments behind this one
    const int count = (p.len + a.cut.seg - 1) / a.cut.seg;
    fold_segments<true, NW>(a, unit - p.index, p.index + 1, count, strip, cn, lane, run, own, &s_map[0][0][0][0], e);
    parity = 1;
  }
  for (int t0 = t_last; p.begin < p.end && t0 >= p.begin; t0 -= TILE) {
    const int mine = p.end - (t0 + run * R);
    Vec8<T> rv[R], rw[R];
    float al[R][8], z[R][8], d[R][8], A[8], H[8], L[8], XA[8], XH[8], XB[8], XL[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) A[c] = H[c] = L[c] = XH[c] = XL[c] = 0.f, XA[c] = XB[c] = 1.f;
    float h = hnext;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float w[8], g[8];
      rv[i] = r.x[0][i];
      rv[i].to_float(z[i]);
      r.x[1][i].to_float(g);
      r.x[2][i].to_float(d[i]);
      if constexpr (GATE) {
        rw[i] = r.x[3][i];
        rw[i].to_float(w);
      }
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
    if (t0 > p.begin) load(t0 - TILE);
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
    float xin = h, yin = e;
#pragma unroll
    for (int u = 0; u < NW; ++u) {
      if (u == wave) xin = h;
      h = fmaf(s_map[parity][0][u][own], h, s_map[parity][1][u][own]);
    }
#pragma unroll
    for (int u = NW - 1; u >= 0; --u) {
      if (u == wave) yin = e;
      e = fmaf(s_map[parity][0][u][own], e, s_map[parity][2][u][own]);
    }
    s_in[0][wave][own] = xin;
    s_in[1][wave][own] = yin;
    float x[8], y[8];  // the state before this lane's run, the gradient behind it
    load8f(&s_in[0][wave][cg * 8], x);
    load8f(&s_in[1][wave][cg * 8], y);
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
    const long at0 = out + (long)t0 * a.D;
#pragma unroll
    for (int i = R - 1; i >= 0; --i) {
      float v[8], w[8], gv[8], gg[8], gw[8];
      rv[i].to_float(v);
      if constexpr (GATE) rw[i].to_float(w);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float dt = d[i][c] + y[c];
        y[c] = al[i][c] * dt;
        gv[c] = GATE ? dt * w[c] : dt;
        gw[c] = dt * v[c];
        gg[c] = y[c] * before[i][c];
      }
      if (i < mine) {
        const unsigned at = (unsigned)__umul24(run * R + i, a.D);
        cn.template store<MODE>((T*)b.dv + at0 + at, gv);
        cn.template store<MODE>((T*)b.dg + at0 + at, gg);
        if constexpr (GATE) cn.template store<MODE>((T*)b.dw + at0 + at, gw);
      }
    }
  }
  if (b.d_s0 != nullptr && p.begin == 0 && wave == 0 && owned < a.D) b.d_s0[(long)p.n * a.D + och] = e;
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
  if (!packed) return (long)B * ((T + kStateTokens - 1) / kStateTokens);
  const long slots = (long)T / kStateTokens + N;
  return slots == 0 && T > 0 ? 1 : slots;  // rows without sequences: the states' pointer says that this is training
}

// A unit takes a workgroup for each of its strips. Uncut, units are sequences: with few of them most of
// the card stands idle; cut, the inputs are read once more (up to 6 of 8 + 6 bytes an element forward, see
// the passes above; 4 of 14 + 4 backward). Measured at 2048 channels in bf16, 4096 tokens, forward (nothing
// is forgotten) and backward in us:
//   sequences                 1          2          3          4          5
//   uncut                 69, 140    69, 141    72, 146    77, 150    86, 158
//   cut                   24,  31    43,  60    64,  91    85, 113   119, 150
// and of 6 the backward 170 uncut, 175 cut. Where workgroups run past a whole round of the card (9
// sequences, 288: 80 and 145 uncut, 84 and 120 cut) the last round counts like a full one: cut where less
// than 0.44 (0.66) of the rounds is used. Units fill the card with four workgroups of 4 waves a compute
// unit. A forward whose fair share of one workgroup of 8 waves a compute unit is 1024 tokens or more takes
// that, and two passes of the outputs (see above; with resets, without, nothing forgotten, against a pass for
// the maps: segments of 512 tokens, 1 x 4096, 24, 27, 28 against 24; of 1024, 2 x 4096, 34, 45, 45 against 43;
// of 1536, 3 x 4096, 57, 64, 64 against 67; of 2048, 1 x 16384, 69, 83, 92 against 86). Packed batches, whose
// lengths the host does not know, are cut at four times the fair share in any case, for a sequence much
// longer than the others.
RecurrenceCut recurrence_cut(bool backward, bool packed, int B, int T, int D, int N) {
  constexpr int TILE = 128;
  RecurrenceCut c{};
  const long strips = strips_of(D), tokens = (long)B * T, groups = N * strips;
  c.seg = T > 0 ? T : 1;
  c.per_sequence = 1;
  c.units = N;
  if (T < (backward ? 3 : 6) * TILE || N == 0 || N > kMaxGroups) return c;
  const long rounds = (groups + 255) / 256;
  const bool few = groups * 100 < rounds * 256 * (backward ? 66 : 44);
  if (!few && !packed) return c;
  const auto share = [&](long of) { return ((tokens * strips + of - 1) / of + TILE - 1) / TILE * TILE; };
  c.twice = !backward && few && share(256) >= 1024;
  long seg = share(c.twice || !few ? 256 : 1024);
  if (seg < 2 * TILE) seg = 2 * TILE;
  if (seg >= T) return c;
  c.cut = true;
  c.seg = (int)seg;
  c.per_sequence = packed ? 1 : (int)((T + seg - 1) / seg);
  c.units = packed ? (int)(T / seg) + N : N * c.per_sequence;
  return c;
}
long recurrence_groups(const RecurrenceCut& c, int D) { return ((long)c.units + 1) * strips_of(D) + 7; }
size_t recurrence_workspace_bytes(const RecurrenceCut& c, int D) {
  return c.cut ? (size_t)c.units * (2 * D + strips_of(D)) * sizeof(float) : 0;
}

namespace {

// Eight waves a workgroup (twice the tile) for whole sequences of up to two workgroups a compute unit:
// 4 x 4096 tokens of 2048 channels 85 -> 76 us forward, 171 -> 150 backward; 64 x 256 53 -> 59. (The
// backward in fp32 has no registers for it.)
bool wide_groups(const RecurrenceCut& c, int strips) { return !c.cut && (long)c.units * strips <= 512; }

// Whether rows begin at lines of 128 bytes.
bool at_lines(const void* p, long stride, size_t size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 128 == 0 && stride * size % 128 == 0);
}
// Inputs of more than half the Infinity Cache (256 MB) are read past the caches: 8 x 2048 tokens of
// 2048 channels in bf16 60 -> 57 us; of half as many, where repeated calls find them there, 26 -> 30.
// (Rows that share lines lose by it: 7 packed sequences of 520 channels in fp32 29 -> 37, and their
// backward by stores past the caches, 8 x 1024 x 1000 in bf16 42 -> 51.) A forward in two passes,
// which reads them twice, does so from the whole cache on: 16384 tokens of 2048 channels 73 -> 69.
bool streamed(const RecurrenceArgs& a, long tokens, int arrays, size_t size, long limit = 128) {
  return tokens * a.D * arrays * (long)size > limit << 20;
}
unsigned grid_of(const RecurrenceArgs& a, int units) {
  const long n = (long)units * strips_of(a.D);
  return (unsigned)(a.shared_lines ? (n + 7) / 8 * 8 : n);
}

template <typename T, bool GATE, int MODE>
void launch_forward(const RecurrenceArgs& a) {
  const hipStream_t st = (hipStream_t)a.stream;
  const dim3 grid(grid_of(a, a.cut.units + a.zero_rest));
  if (a.cut.cut && a.cut.twice) {  // what the first pass reads through the caches, the second finds there in part
    constexpr int FIRST = MODE == kStream ? kLines : MODE;
    hipLaunchKernelGGL((gdn2_recurrence_kernel<T, GATE, 8, FIRST, kFirst>), grid, dim3(512), 0, st, a);
    hipLaunchKernelGGL((gdn2_recurrence_kernel<T, GATE, 8, MODE, kSecond>), dim3(grid_of(a, a.cut.units)), dim3(512), 0, st, a);
  } else if (wide_groups(a.cut, strips_of(a.D))) {
    hipLaunchKernelGGL((gdn2_recurrence_kernel<T, GATE, 8, MODE, kWhole>), grid, dim3(512), 0, st, a);
  } else {
    hipLaunchKernelGGL((gdn2_recurrence_kernel<T, GATE, 4, MODE, kWhole>), grid, dim3(256), 0, st, a);
  }
}
template <typename T, bool GATE>
hipError_t forward(RecurrenceArgs a) {
  const long tokens = a.cu_seqlens != nullptr ? a.T : (long)a.N * a.T;
  a.zero_rest = a.cu_seqlens != nullptr && a.states != nullptr && a.o != nullptr;
  a.shared_lines = !at_lines(a.v, a.v_stride, sizeof(T)) || !at_lines(a.g, a.g_stride, sizeof(T)) ||
                   !at_lines(a.w, a.w_stride, sizeof(T)) || !at_lines(a.o, a.D, sizeof(T));
  if (a.cut.cut && !a.cut.twice)
    hipLaunchKernelGGL((gdn2_recurrence_maps_kernel<T, GATE, false>), dim3(grid_of(a, a.cut.units)), dim3(256), 0,
                       (hipStream_t)a.stream, a, (const T*)nullptr);
  if (a.shared_lines) launch_forward<T, GATE, kSharedLines>(a);
  else if (streamed(a, tokens, GATE ? 3 : 2, sizeof(T), a.cut.cut && a.cut.twice ? 256 : 128)) launch_forward<T, GATE, kStream>(a);
  else launch_forward<T, GATE, kLines>(a);
  return hipGetLastError();
}

template <typename T, bool GATE, int MODE>
void launch_backward(const RecurrenceBwdArgs& b) {
  const hipStream_t st = (hipStream_t)b.f.stream;
  const dim3 grid(grid_of(b.f, b.f.cut.units + b.f.zero_rest));
  if constexpr (sizeof(T) == 2) {
    if (wide_groups(b.f.cut, strips_of(b.f.D))) {
      hipLaunchKernelGGL((gdn2_recurrence_bwd_kernel<T, GATE, 8, MODE>), grid, dim3(512), 0, st, b);
      return;
    }
  }
  hipLaunchKernelGGL((gdn2_recurrence_bwd_kernel<T, GATE, 4, MODE>), grid, dim3(256), 0, st, b);
}
template <typename T, bool GATE>
hipError_t backward(RecurrenceBwdArgs b) {
  RecurrenceArgs& a = b.f;
  const long tokens = a.cu_seqlens != nullptr ? a.T : (long)a.N * a.T;
  a.zero_rest = a.cu_seqlens != nullptr;
  a.shared_lines = !at_lines(a.v, a.v_stride, sizeof(T)) || !at_lines(a.g, a.g_stride, sizeof(T)) ||
                   !at_lines(a.w, a.w_stride, sizeof(T)) || !at_lines(b.d_o, a.D, sizeof(T));
  if (a.cut.cut)
    hipLaunchKernelGGL((gdn2_recurrence_maps_kernel<T, false, true>), dim3(grid_of(a, a.cut.units)), dim3(256), 0,
                       (hipStream_t)a.stream, a, (const T*)b.d_o);
  if (a.shared_lines) launch_backward<T, GATE, kSharedLines>(b);
  else if (streamed(a, tokens, GATE ? 4 : 3, sizeof(T))) launch_backward<T, GATE, kStream>(b);
  else launch_backward<T, GATE, kLines>(b);
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
