// Verification of drafted tokens on gfx950, from given random numbers u in [0, 1):
//     draft i is accepted where u_i q_i(x_i) < p_i(x_i) and all before it are;   a: their number
//     weights  m_j = max(p_a(j) - q_a(j), 0)  at a rejected draft (p_a itself where all are zero),
//              m_j = p_a(j)  behind the last draft
//     token = the first j with  m_0 + .. + m_j > u_L (m_0 + .. + m_{V-1}).
// Drafts that were certain (no q) have q(x_i) = 1 and nothing elsewhere. Values that are not
// positive, NaN among them, count as zero.
//
// The token is a border in a sum over the vocabulary, so products, differences and sums are in
// fp64: those of fp32 values are exact or rounded at 2^-53, and no order of a sum moves a border
// that a draw meets. Bound by HBM: one row of p and one of q are read (8 V bytes a sequence in
// fp32). The first kernel leaves the sums of pieces of kPiece entries, many workgroups a row; the
// second finds the piece that holds the border and reads that one again.

#include "gdn2_attn_device.h"
#include "gdn2_stack_launch.h"

namespace gdn2 {

namespace {

constexpr int kPiece = 4096;  // vocabulary entries of a piece: 16 a lane

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

__device__ __forceinline__ double positive(double x) { return x > 0 ? x : 0; }

// Accepted drafts of sequence n and the drafts it has, in every lane of the wave.
template <typename T>
__device__ __forceinline__ void accepted(const VerifyArgs& a, int n, int& taken, int& length) {
  const int lane = threadIdx.x & 63;
  length = a.draft_len != nullptr ? scalar_load(a.draft_len, n) : a.L;
  length = length < 0 ? 0 : length > a.L ? a.L : length;
  taken = 0;
  for (int i0 = 0; i0 < length; i0 += 64) {
    const int i = i0 + lane;
    bool ok = false;
    if (i < length) {
      const int x = a.drafts[(long)n * a.L + i];
      if (x >= 0 && x < a.V) {
        const double p = to_f(((const T*)a.p)[((long)n * (a.L + 1) + i) * a.V + x]);
        const double q = a.q != nullptr ? (double)to_f(((const T*)a.q)[((long)n * a.L + i) * a.V + x]) : 1.0;
        ok = (double)a.u[(long)n * (a.L + 1) + i] * positive(q) < p;
      }
    }
    const uint64_t yes = __ballot(ok);
    const int run = yes == ~0ull ? 64 : __builtin_ctzll(~yes);
    taken += run;
    if (run < 64) break;
  }
  taken = __builtin_amdgcn_readfirstlane(taken);
}

// Eight entries at j of a row that may start anywhere, as far as the row goes (zeros behind).
template <typename T>
__device__ __forceinline__ void entries(const T* row, int j, int V, float* f) {
  typedef T vec __attribute__((ext_vector_type(8)));
  typedef vec loose __attribute__((aligned(sizeof(T))));
  if (j + 8 <= V) {
    const vec v = *reinterpret_cast<const loose*>(row + j);
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = to_f(v[c]);
  } else {
#pragma unroll
    for (int c = 0; c < 8; ++c) f[c] = j + c < V ? to_f(row[j + c]) : 0.f;
  }
}

// The rows that a sequence draws from.
template <typename T>
struct Rows {
  const T *p, *q;  // q null: nothing is subtracted
  int gone;        // a certain draft that was rejected: its entry counts as zero (-1: none)
};
template <typename T>
__device__ __forceinline__ Rows<T> rows_of(const VerifyArgs& a, int n, int taken, int length) {
  Rows<T> r;
  r.p = (const T*)a.p + ((long)n * (a.L + 1) + taken) * a.V;
  const bool rejected = taken < length;
  r.q = rejected && a.q != nullptr ? (const T*)a.q + ((long)n * a.L + taken) * a.V : nullptr;
  r.gone = rejected && a.q == nullptr ? scalar_load(a.drafts, (long)n * a.L + taken) : -1;
  return r;
}
// Weights of the entries j .. j + 7, and p itself.
template <typename T>
__device__ __forceinline__ void weights(const Rows<T>& r, int j, int V, double* m, double* p) {
  float x[8], y[8];
  entries(r.p, j, V, x);
  if (r.q != nullptr) entries(r.q, j, V, y);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    p[c] = positive(x[c]);
    m[c] = r.q != nullptr ? positive(p[c] - positive(y[c])) : j + c == r.gone ? 0.0 : p[c];
  }
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(256) gdn2_verify_sums_kernel(VerifyArgs a, int pieces) {
  __shared__ double s[2][4];
  const int n = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int taken, length;
  accepted<T>(a, n, taken, length);
  const Rows<T> r = rows_of<T>(a, n, taken, length);
  double sm = 0, sp = 0;
#pragma unroll
  for (int k = 0; k < kPiece / 2048; ++k) {
    double m[8], p[8];
    weights(r, piece * kPiece + k * 2048 + threadIdx.x * 8, a.V, m, p);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      sm += m[c];
      sp += p[c];
    }
  }
  sm = wave_sum64(sm);
  sp = wave_sum64(sp);
  if (lane == 0) {
    s[0][wave] = sm;
    s[1][wave] = sp;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* t = s[threadIdx.x];
    a.sums[(long)blockIdx.x * 2 + threadIdx.x] = (t[0] + t[1]) + (t[2] + t[3]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) gdn2_verify_token_kernel(VerifyArgs a, int pieces) {
  __shared__ double s_wave[4];
  __shared__ int s_first[4], s_some[4];
  const int n = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int taken, length;
  accepted<T>(a, n, taken, length);
  const Rows<T> r = rows_of<T>(a, n, taken, length);
  const double* sums = a.sums + (long)n * pieces * 2;
  // every wave by itself: the total, then the piece whose sums pass the border
  double tm = 0, tp = 0;
  for (int i = lane; i < pieces; i += 64) {
    tm += sums[2 * i];
    tp += sums[2 * i + 1];
  }
  tm = wave_sum64(tm);
  tp = wave_sum64(tp);
  const bool plain = !(tm > 0);  // nothing is left of p: p itself
  const double total = plain ? tp : tm;
  const double border = (double)a.u[(long)n * (a.L + 1) + a.L] * total;
  int piece = -1;      // the one that holds the border
  double before = 0;   // the sum in front of it
  int last = -1;       // the last piece that holds anything
  double sum = 0, last_before = 0;
  for (int i0 = 0; i0 < pieces && piece < 0; i0 += 64) {
    const int i = i0 + lane;
    const double x = i < pieces ? sums[2 * i + plain] : 0;
    double c = x;  // inclusive over the lanes
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double y = __shfl_up(c, m, 64);
      if (lane >= m) c += y;
    }
    c += sum;
    const uint64_t hit = __ballot(x > 0 && c > border), some = __ballot(x > 0);
    if (hit) {
      const int k = __builtin_ctzll(hit);
      piece = i0 + k;
      before = k > 0 ? __shfl(c, k - 1, 64) : sum;
    }
    if (some) {
      const int k = 63 - __builtin_clzll(some);
      last = i0 + k;
      last_before = k > 0 ? __shfl(c, k - 1, 64) : sum;
    }
    sum = __shfl(c, 63, 64);
  }
  if (piece < 0) {  // a border at or past the end (u of 1): the last entry that holds anything
    piece = last;
    before = last_before;
  }
  int token = -1;
  if (piece >= 0) {
    // the piece again, in order: lane t of the workgroup holds entries 16 t .. 16 t + 15
    double m[16], own = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      double p[8];
      weights(r, piece * kPiece + threadIdx.x * 16 + k * 8, a.V, m + 8 * k, p);
      if (plain)
#pragma unroll
        for (int c = 0; c < 8; ++c) m[8 * k + c] = p[c];
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) own += m[c];
    double c = own;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      const double y = __shfl_up(c, k, 64);
      if (lane >= k) c += y;
    }
    if (lane == 63) s_wave[wave] = c;
    __syncthreads();
    double front = before + (c - own);
#pragma unroll
    for (int u = 0; u < 3; ++u)
      if (u < wave) front += s_wave[u];
    // the first entry past the border; where rounding leaves none, the last that holds anything
    int first = 1 << 30, some = -1;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      front += m[k];
      const int j = piece * kPiece + threadIdx.x * 16 + k;
      if (m[k] > 0) {
        some = j;
        if (front > border && first == 1 << 30) first = j;
      }
    }
#pragma unroll
    for (int k = 32; k > 0; k >>= 1) {
      const int f = __shfl_xor(first, k, 64), l = __shfl_xor(some, k, 64);
      first = f < first ? f : first;
      some = l > some ? l : some;
    }
    if (lane == 0) {
      s_first[wave] = first;
      s_some[wave] = some;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      first = s_first[u] < first ? s_first[u] : first;
      some = s_some[u] > some ? s_some[u] : some;
    }
    token = first < 1 << 30 ? first : some;
  }
  for (int i = threadIdx.x; i <= a.L; i += 256)
    a.tokens[(long)n * (a.L + 1) + i] = i < taken ? a.drafts[(long)n * a.L + i] : i == taken ? token : -1;
  if (threadIdx.x == 0) a.commit[n] = taken + 1;
}

int verify_pieces(int V) { return (V + kPiece - 1) / kPiece; }

template <typename T>
static hipError_t verify(const VerifyArgs& a) {
  const int pieces = verify_pieces(a.V);
  const hipStream_t st = (hipStream_t)a.stream;
  hipLaunchKernelGGL((gdn2_verify_sums_kernel<T>), dim3((unsigned)((long)pieces * a.N)), dim3(256), 0, st, a, pieces);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((gdn2_verify_token_kernel<T>), dim3((unsigned)a.N), dim3(256), 0, st, a, pieces);
  return hipGetLastError();
}

hipError_t launch_verify(const VerifyArgs& a) {
  return a.dtype == 0 ? verify<bf16>(a) : verify<float>(a);
}

}  // namespace gdn2
