// Verification of drafted tokens on gfx950, from given random numbers u in [0, 1):
//     draft i is accepted where u_i q_i(x_i) < p_i(x_i) and all before it are;   a: their number
//     weights  m_j = max(p_a(j) - q_a(j), 0)  at a rejected draft (p_a itself where all are zero),
//              m_j = p_a(j)  behind the last draft
//     token = the first j with  m_0 + .. + m_j > u_L (m_0 + .. + m_{V-1}).
// Drafts that were certain (no q) have q(x_i) = 1 and nothing elsewhere. Values that are not
// positive, NaN among them, count as zero.
//
// The token is a border in a sum over the vocabulary, so products, differences and sums are in
// fp64. Those of fp32 values are exact, or rounded at 2^-53 where exponents lie more than 29 bits apart or
// the row is long: a border is then known to within some 2^-53 of the total, as is u times it, and a draw
// that near to one may give the neighbouring entry that holds anything. Equal inputs give equal tokens (the
// orders of the sums are fixed). Bound by HBM where sequences are many (one row of p and one of q are read, 8 V
// bytes a sequence in fp32: 64 of 131071 entries 12 us, 5.4 TB/s), by the latency of dependent loads
// where they are few. The first kernel leaves the sums of pieces of kPiece entries, many workgroups a
// row; the second finds the piece that holds the border and reads that one again (5 us). One
// workgroup a sequence for all of it measured 7.7 us against 8.1 at 1000 entries, 12 against 8.4 at
// 32000, 26 against 8.2 at 131071, and 46 against 47 for 256 sequences of 131071.

#include "gdn2_attn_device.h"
#include "gdn2_stack_launch.h"

namespace gdn2 {

namespace {

constexpr int kPiece = 4096;  // vocabulary entries of a piece

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// Accepted drafts of sequence n and the drafts it has, in every lane of the wave. (The first round's
// loads do not wait for the number of drafts.)
template <typename T>
__device__ __forceinline__ void accepted(const VerifyArgs& a, int n, int& taken, int& length) {
  const int lane = threadIdx.x & 63;
  length = a.draft_len != nullptr ? a.draft_len[n] : a.L;
  taken = 0;
  for (int i0 = 0; i0 < a.L; i0 += 64) {
    const int i = i0 + lane;
    bool ok = false;
    if (i < a.L) {
      const int x = a.drafts[(long)n * a.L + i];
      const float u = a.u[(long)n * (a.L + 1) + i];
      if (x >= 0 && x < a.V) {
        const float p = to_f(((const T*)a.p)[((long)n * (a.L + 1) + i) * a.V + x]);
        const float q = a.q != nullptr ? to_f(((const T*)a.q)[((long)n * a.L + i) * a.V + x]) : 1.f;
        ok = (double)u * (double)fmaxf(q, 0.f) < (double)p;
      }
    }
    const uint64_t yes = __ballot(ok && i < length);
    const int run = yes == ~0ull ? 64 : __builtin_ctzll(~yes);
    taken += run;
    if (run < 64) break;
  }
  taken = uniform(taken);
  length = uniform(length > a.L ? a.L : length);
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
  r.gone = rejected && a.q == nullptr ? uniform(a.drafts[(long)n * a.L + taken]) : -1;
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
    m[c] = p[c] = fmaxf(x[c], 0.f);  // a NaN gives the other operand
    if (r.q != nullptr) m[c] = fmax(p[c] - (double)fmaxf(y[c], 0.f), 0.0);
    if (j + c == r.gone) m[c] = 0;
  }
}

// Sum of the weights of [begin, end) over a wave, lanes taking 8 entries in turn; whole: that of p.
template <typename T>
__device__ __forceinline__ double wave_weights(const Rows<T>& r, int begin, int end, int V, double& whole) {
  double sum = 0, all = 0;
#pragma unroll 4
  for (int j = begin + (threadIdx.x & 63) * 8; j < end; j += 512) {
    double m[8], p[8];
    weights(r, j, V, m, p);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      sum += m[c];
      all += p[c];
    }
  }
  whole = wave_sum64(all);
  return wave_sum64(sum);
}

// The first of n sums (a lane reads sum(i), n <= 64) whose running total from `sum` on passes the
// border: its index, and the total in front of it; -1 where none does. last, last_front: the last sum
// that is not zero. Every lane gets them; sum ends at the total.
struct Found {
  int at = -1, last = -1;
  double front = 0, last_front = 0;
};
__device__ __forceinline__ void find_sum(double x, int i0, double border, double& sum, Found& f) {
  const int lane = threadIdx.x & 63;
  double c = x;  // inclusive over the lanes
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const double y = __shfl_up(c, m, 64);
    if (lane >= m) c += y;
  }
  c += sum;
  const uint64_t hit = __ballot(x > 0 && c > border), some = __ballot(x > 0);
  if (hit && f.at < 0) {
    const int k = __builtin_ctzll(hit);
    f.at = i0 + k;
    f.front = k > 0 ? __shfl(c, k - 1, 64) : sum;
  }
  if (some) {
    const int k = 63 - __builtin_clzll(some);
    f.last = i0 + k;
    f.last_front = k > 0 ? __shfl(c, k - 1, 64) : sum;
  }
  sum = __shfl(c, 63, 64);
}

// Of a piece's entries, which begin at `base` with the sum `front` before them: the first that passes
// the border, else the last that holds anything. For a workgroup of 4 waves, 16 entries a lane.
template <typename T>
__device__ __forceinline__ int locate(const Rows<T>& r, int base, int V, bool plain, double border, double front) {
  constexpr int WAVES = 4, PER = kPiece / (64 * WAVES);
  __shared__ double s_wave[WAVES];
  __shared__ int s_first[WAVES], s_some[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double m[PER], own = 0;
#pragma unroll
  for (int k = 0; k < PER; k += 8) {
    double p[8];
    weights(r, base + (int)threadIdx.x * PER + k, V, m + k, p);
    if (plain)
#pragma unroll
      for (int c = 0; c < 8; ++c) m[k + c] = p[c];
  }
#pragma unroll
  for (int c = 0; c < PER; ++c) own += m[c];
  double c = own;
#pragma unroll
  for (int k = 1; k < 64; k <<= 1) {
    const double y = __shfl_up(c, k, 64);
    if (lane >= k) c += y;
  }
  if (lane == 63) s_wave[wave] = c;
  __syncthreads();
  double at = front + (c - own);
#pragma unroll
  for (int u = 0; u < WAVES; ++u)
    if (u < wave) at += s_wave[u];
  int first = 1 << 30, last = -1;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    at += m[k];
    if (m[k] > 0) {
      last = base + (int)threadIdx.x * PER + k;
      if (at > border && first == 1 << 30) first = last;
    }
  }
  const uint64_t hit = __ballot(first < 1 << 30), any = __ballot(last >= 0);
  first = hit ? __shfl(first, __builtin_ctzll(hit), 64) : 1 << 30;
  last = any ? __shfl(last, 63 - __builtin_clzll(any), 64) : -1;
  if (lane == 0) {
    s_first[wave] = first;
    s_some[wave] = last;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < WAVES; ++u) {
    first = s_first[u] < first ? s_first[u] : first;
    last = s_some[u] > last ? s_some[u] : last;
  }
  return first < 1 << 30 ? first : last;
}

}  // namespace

// The sums of a piece; the first piece's workgroup also says how many drafts were accepted.
template <typename T>
__global__ void __launch_bounds__(256) gdn2_verify_sums_kernel(VerifyArgs a, int pieces) {
  __shared__ double s[2][4];
  const int n = blockIdx.x / pieces, piece = blockIdx.x % pieces;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int taken, length;
  accepted<T>(a, n, taken, length);
  const Rows<T> r = rows_of<T>(a, n, taken, length);
  const int begin = piece * kPiece + wave * (kPiece / 4), end = begin + kPiece / 4 < a.V ? begin + kPiece / 4 : a.V;
  double whole;
  const double sum = wave_weights(r, begin, end, a.V, whole);
  if (lane == 0) {
    s[0][wave] = sum;
    s[1][wave] = whole;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* t = s[threadIdx.x];
    a.sums[(long)blockIdx.x * 2 + threadIdx.x] = (t[0] + t[1]) + (t[2] + t[3]);
  }
  if (piece == 0 && threadIdx.x == 0) a.commit[n] = taken + 1;
}

template <typename T>
__global__ void __launch_bounds__(256) gdn2_verify_token_kernel(VerifyArgs a, int pieces) {
  const int n = blockIdx.x, lane = threadIdx.x & 63;
  const double u = a.u[(long)n * (a.L + 1) + a.L];
  const int taken = uniform(a.commit[n]) - 1;  // the first kernel's
  const int length = uniform(a.draft_len != nullptr && a.draft_len[n] < a.L ? a.draft_len[n] : a.L);
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
  const double border = u * (plain ? tp : tm);
  Found f;
  double all = 0;
  for (int i0 = 0; i0 < pieces && f.at < 0; i0 += 64)
    find_sum(i0 + lane < pieces ? sums[2 * (i0 + lane) + plain] : 0, i0, border, all, f);
  const int at = f.at >= 0 ? f.at : f.last;  // a border at or past the end: the last entry that holds anything
  const int token = at >= 0 ? locate(r, at * kPiece, a.V, plain, border, f.at >= 0 ? f.front : f.last_front) : -1;
  for (int i = threadIdx.x; i <= a.L; i += 256)
    a.tokens[(long)n * (a.L + 1) + i] = i < taken ? a.drafts[(long)n * a.L + i] : i == taken ? token : -1;
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
