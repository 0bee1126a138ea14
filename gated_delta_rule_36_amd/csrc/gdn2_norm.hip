// The norm between the layers of a stack on gfx950, with the residual's addition:
//     h = x + r          (stored in r's type: the stream that the next layer adds to)
//     y = h rho weight,  rho = 1 / sqrt(mean(h^2) + eps)   (of h as it is stored)
// y in x's type, or in 8 bits for the next projection: e4m3 codes with one power-of-two scale for
// every group of channels, the smallest s >= 2^-64 with max|y| <= 448 s. And the gradients, with
// u = dy weight and n = h rho:
//     dh_total = dh + rho (u - n mean(u n)) = dx = dr,   dweight = sum over rows of dy n.
//
// Bound by HBM: every row is read once and kept in registers between the sum and the output. Sums over a
// row are in fp64, whose exponent holds the square of any fp32 value and the product of any two; rho and
// mean(u n) are back in fp32's range where the row's root mean square is. (Against fp32 sums: forward the same
// times, backward 28.4 -> 29.1 us at 65536 rows of 256, 123 -> 127 at 2048 rows of 16384, else the same.)

#include "gdn2_attn_device.h"
#include "gdn2_stack_device.h"
#include "gdn2_stack_launch.h"

namespace gdn2 {

namespace {

// Sum over the LANES lanes of a row.
template <int LANES, typename T>
__device__ __forceinline__ T lanes_sum(T x) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) x += __shfl_xor(x, m, 64);
  return x;
}

// Sums over a row of K values: LANES lanes of a wave, and W waves through LDS (s: of this call's own).
template <int LANES, int W, int K, typename T>
__device__ __forceinline__ void row_total(T (&x)[K], T (*s)[W], int wave) {
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lanes_sum<LANES>(x[k]);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) s[k][wave] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = 0;
#pragma unroll
      for (int u = 0; u < W; ++u) x[k] += s[k][u];
    }
    __syncthreads();
  }
}

// 1 / sqrt(x) to fp32's precision of an x whose exponent may lie far outside fp32's (four powers of two at a
// time into 0.5 .. 2, and back).
__device__ __forceinline__ float rsqrt_of(double x) {
  const int k = __builtin_amdgcn_frexp_exp(x) >> 1;  // 0, infinity, NaN: 0
  return ldexpf(rsqrtf((float)ldexp(x, -2 * k)), -k);
}

// 2^k with the smallest k in [-64, 126] for which amax <= 448 * 2^k; NaN and zero give 2^-64.
__device__ __forceinline__ float power_scale(double amax) {
  if (!(amax > 0)) return __uint_as_float((127 - 64) << 23);
  const uint64_t bits = __builtin_bit_cast(uint64_t, amax);
  int e = (int)(bits >> 52) - 1022;  // amax = m 2^e, m in [0.5, 1) (doubles: never subnormal here)
  const bool high = (bits & ((1ull << 52) - 1)) > 0xC000000000000ull;  // m > 0.875
  e = e - (high ? 8 : 9);
  e = e < -64 ? -64 : e > 126 ? 126 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ double lanes_max(double x, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) {
    const double y = __shfl_xor(x, m, 64);
    x = x > y || x != x ? x : y;  // a NaN stays
  }
  return x;
}

__device__ __forceinline__ uint32_t e4m3x4(const float* f) {
  const int r = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], r, true);
}

}  // namespace

// A row belongs to LANES lanes of a wave or (LANES = 64) to W waves, which hold E steps of 8 channels a
// lane. BITS8: the output in 8 bits. There the groups' maxima are in fp64 as well (h and weight are exact in
// it, so is their product): the scale steps where a maximum passes 448 times a power of two, and must not
// step by a rounding.
template <typename T, typename TR, int LANES, int E, int W, bool ADD, bool BITS8>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) gdn2_residual_norm_kernel(ResidualNormArgs a) {
  __shared__ double s_sum[1][W];
  const int lane = threadIdx.x & 63, in_row = lane % LANES;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long row = W == 1 ? ((long)blockIdx.x * 4 + wave) * (64 / LANES) + lane / LANES : (long)blockIdx.x;
  if (W == 1 && row >= a.rows) return;
  const int part = W == 1 ? 0 : wave;
  const T* x = (const T*)a.x + row * a.x_stride;
  const TR* r = ADD ? (const TR*)a.r + row * a.r_stride : nullptr;
  Vec8<T> rx[E];
  Vec8<TR> rr[E];
  if (a.stream_rows) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) {
        load_stream(rx[e], x + ch);
        if constexpr (ADD) load_stream(rr[e], r + ch);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) {
        rx[e].load(x + ch);
        if constexpr (ADD) rr[e].load(r + ch);
      }
    }
  }
  float h[E][8];
  double sum[1] = {0};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int ch = ((e * W + part) * LANES + in_row) * 8;
    if (ch < a.D) {
      rx[e].to_float(h[e]);
      if constexpr (ADD) {
        float f[8];
        rr[e].to_float(f);
#pragma unroll
        for (int c = 0; c < 8; ++c) h[e][c] = to_f(from_f<TR>(h[e][c] + f[c]));
        store8((TR*)a.h + row * a.D + ch, h[e]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < 8; ++c) h[e][c] = 0.f;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) sum[0] += (double)h[e][c] * (double)h[e][c];
  }
  row_total<LANES, W>(sum, s_sum, wave);
  const double ms = sum[0] / a.D + (double)a.eps;
  if constexpr (!BITS8) {
    const float rho = rsqrt_of(ms);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) {
        const f4 w0 = reinterpret_cast<const f4*>(a.weight + ch)[0], w1 = reinterpret_cast<const f4*>(a.weight + ch)[1];
        float y[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) y[c] = h[e][c] * rho * (c < 4 ? w0[c] : w1[c - 4]);
        store8((T*)a.y + row * a.D + ch, y);
      }
    }
  } else {
    const double rho = 1.0 / sqrt(ms);
    const float rho32 = (float)rho;
    const bool whole = a.group >= a.D;  // one scale a row
    const int lanes = a.group / 8;  // of a group
    double big[E], most = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      big[e] = 0;
      if (ch < a.D) {
        const f4 w0 = reinterpret_cast<const f4*>(a.weight + ch)[0], w1 = reinterpret_cast<const f4*>(a.weight + ch)[1];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float w = c < 4 ? w0[c] : w1[c - 4];
          const double p = fabs((double)h[e][c] * (double)w);
          big[e] = big[e] > p || big[e] != big[e] ? big[e] : p;
          h[e][c] = h[e][c] * rho32 * w;
        }
      }
      most = most > big[e] || most != most ? most : big[e];
    }
    if (whole) {
      most = lanes_max(most, LANES);
      if constexpr (W > 1) {
        if (lane == 0) s_sum[0][wave] = most;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const double y = s_sum[0][u];
          most = most > y || most != most ? most : y;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      const float s = power_scale((whole ? most : lanes_max(big[e], lanes)) * rho);
      if (ch < a.D) {
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));  // 1 / s, exact
        float f[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) f[c] = h[e][c] * inv;
        *reinterpret_cast<uint2*>((uint8_t*)a.y + row * a.D + ch) = make_uint2(e4m3x4(f), e4m3x4(f + 4));
        if (ch % a.group == 0) a.scale[row * (a.D / a.group) + ch / a.group] = s;
      }
    }
  }
}

// Gradients. A wave (or workgroup) walks rows and keeps its part of the weight's gradient in
// registers; each workgroup leaves one partial sum, which the second kernel adds in a fixed order.
template <typename T, typename TR, int LANES, int E, int W, bool DH>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) gdn2_residual_norm_bwd_kernel(ResidualNormBwdArgs a) {
  constexpr int ROWS = W == 1 ? 4 * (64 / LANES) : 1;  // of a workgroup at a time
  __shared__ __attribute__((aligned(16))) float s_part[ROWS][W == 1 ? E * LANES * 8 : 4];
  __shared__ double s_sum[2][W];
  const int lane = threadIdx.x & 63, in_row = lane % LANES;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = W == 1 ? 0 : wave;
  float w[E][8], dw[E][8];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int ch = ((e * W + part) * LANES + in_row) * 8;
#pragma unroll
    for (int c = 0; c < 8; ++c) w[e][c] = dw[e][c] = 0.f;
    if (ch < a.D) {
      const f4 w0 = reinterpret_cast<const f4*>(a.weight + ch)[0], w1 = reinterpret_cast<const f4*>(a.weight + ch)[1];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[e][c] = c < 4 ? w0[c] : w1[c - 4];
    }
  }
  const int mine = W == 1 ? wave * (64 / LANES) + lane / LANES : 0;
  const double per = 1.0 / a.D;
  for (long row = (long)blockIdx.x * ROWS + mine; row < a.rows; row += (long)gridDim.x * ROWS) {
    Vec8<T> rg[E];
    Vec8<TR> rh[E], rd[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) {
        load_stream(rg[e], (const T*)a.dy + row * a.D + ch);
        load_stream(rh[e], (const TR*)a.h + row * a.h_stride + ch);
        if constexpr (DH) load_stream(rd[e], (const TR*)a.dh + row * a.D + ch);
      } else {
        rg[e].zero();
        rh[e].zero();
      }
    }
    double sum[2] = {0, 0};  // h^2, u h
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float g[8], h[8];
      rg[e].to_float(g);
      rh[e].to_float(h);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        sum[0] = fma((double)h[c], (double)h[c], sum[0]);
        sum[1] = fma((double)(g[c] * w[e][c]), (double)h[c], sum[1]);
      }
    }
    row_total<LANES, W>(sum, s_sum, wave);
    const float rho = rsqrt_of(fma(sum[0], per, (double)a.eps));
    const float un = (float)(sum[1] * per * (double)rho);  // mean(u n)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) {
        float g[8], h[8], d[8];
        rg[e].to_float(g);
        rh[e].to_float(h);
        if constexpr (DH) rd[e].to_float(d);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float n = h[c] * rho, t = rho * (g[c] * w[e][c] - n * un);
          dw[e][c] = fmaf(g[c], n, dw[e][c]);
          d[c] = DH ? d[c] + t : t;
        }
        store8((T*)a.dx + row * a.D + ch, d);
        if constexpr (sizeof(T) != sizeof(TR)) store8((TR*)a.dr + row * a.D + ch, d);
      }
    }
  }
  float* const out = a.partial + (long)blockIdx.x * a.D;
  if constexpr (W == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) store8(&s_part[mine][(e * LANES + in_row) * 8], dw[e]);
    __syncthreads();
    for (int ch = threadIdx.x * 4; ch < a.D; ch += 1024) {
      double s[4] = {0, 0, 0, 0};
#pragma unroll
      for (int u = 0; u < ROWS; ++u) {
        const f4 x = *reinterpret_cast<const f4*>(&s_part[u][ch]);
#pragma unroll
        for (int c = 0; c < 4; ++c) s[c] += x[c];
      }
      *reinterpret_cast<f4*>(out + ch) = f4{(float)s[0], (float)s[1], (float)s[2], (float)s[3]};
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int ch = ((e * W + part) * LANES + in_row) * 8;
      if (ch < a.D) store8(out + ch, dw[e]);
    }
  }
}

// The weight's gradient: 32 channels (a line of the partial sums) a workgroup, 32 of its lanes walking
// the sums of each. What several rows' lanes leave is added in fp64, at no cost in time (22684 rows of 64
// channels in fp32: 0.8e-7 off the formula in the 2-norm, 2.0e-7 with all sums in fp32).
__global__ void __launch_bounds__(1024) gdn2_residual_norm_dweight_kernel(const float* partial, float* dweight, int D, int groups) {
  __shared__ double s[32][32];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5, ch = blockIdx.x * 32 + c;
  double x = 0;
  if (ch < D) {
#pragma unroll 16
    for (int g = k; g < groups; g += 32) x += partial[(long)g * D + ch];
  }
  s[k][c] = x;
  __syncthreads();
  if (k == 0 && ch < D) {
    double t = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][c];
    dweight[ch] = (float)t;
  }
}

namespace {

// How a row is laid out. Up to 512 channels it takes no more lanes of a wave than it fills (65536 rows
// of 256 in bf16: 22-24 us, backward 29; with a wave a row 30 and 43); wider ones take a wave up to 2048 channels, unless rows are too few to fill the
// card, and 4 or 8 waves above.
template <int LANES_, int E_, int W_>
struct Layout {
  static constexpr int LANES = LANES_, E = E_, W = W_;
  static constexpr int rows = W == 1 ? 4 * (64 / LANES) : 1;  // of a workgroup
  static constexpr int threads = W == 1 ? 256 : 64 * W;
};
template <typename F>
auto with_layout(long rows, int D, F f) {
  if (D <= 64) return f(Layout<8, 1, 1>());
  if (D <= 128) return f(Layout<16, 1, 1>());
  if (D <= 256) return f(Layout<32, 1, 1>());
  if (D <= 512) return f(Layout<64, 1, 1>());
  if (D <= 2048 && rows >= 1024) return D <= 1024 ? f(Layout<64, 2, 1>()) : f(Layout<64, 4, 1>());
  if (D <= 2048) return f(Layout<64, 1, 4>());
  if (D <= 4096) return f(Layout<64, 2, 4>());
  if (D <= 8192) return f(Layout<64, 4, 4>());
  return f(Layout<64, 4, 8>());
}

template <typename T, typename TR>
hipError_t norm_launch(const ResidualNormArgs& a) {
  return with_layout(a.rows, a.D, [&](auto layout) {
    typedef decltype(layout) L;
    const dim3 grid((unsigned)((a.rows + L::rows - 1) / L::rows)), block(L::threads);
    const hipStream_t st = (hipStream_t)a.stream;
    if (a.scale) {
      if (a.r) hipLaunchKernelGGL((gdn2_residual_norm_kernel<T, TR, L::LANES, L::E, L::W, true, true>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((gdn2_residual_norm_kernel<T, T, L::LANES, L::E, L::W, false, true>), grid, block, 0, st, a);
    } else {
      if (a.r) hipLaunchKernelGGL((gdn2_residual_norm_kernel<T, TR, L::LANES, L::E, L::W, true, false>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((gdn2_residual_norm_kernel<T, T, L::LANES, L::E, L::W, false, false>), grid, block, 0, st, a);
    }
    return hipGetLastError();
  });
}

template <typename T, typename TR>
hipError_t norm_bwd_launch(const ResidualNormBwdArgs& a) {
  const int groups = residual_norm_bwd_groups(a.rows, a.D);
  const hipStream_t st = (hipStream_t)a.stream;
  const hipError_t err = with_layout(a.rows, a.D, [&](auto layout) {
    typedef decltype(layout) L;
    const dim3 grid((unsigned)groups), block(L::threads);
    if (a.dh) hipLaunchKernelGGL((gdn2_residual_norm_bwd_kernel<T, TR, L::LANES, L::E, L::W, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((gdn2_residual_norm_bwd_kernel<T, TR, L::LANES, L::E, L::W, false>), grid, block, 0, st, a);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(gdn2_residual_norm_dweight_kernel, dim3((unsigned)((a.D + 31) / 32)), dim3(1024), 0, st, a.partial, a.dweight, a.D, groups);
  return hipGetLastError();
}

}  // namespace

int residual_norm_bwd_groups(long rows, int D) {
  const long full = with_layout(rows, D, [&](auto layout) { return (rows + decltype(layout)::rows - 1) / decltype(layout)::rows; });
  return (int)(full < 512 ? full : 512);
}

// Inputs of more than half the Infinity Cache (256 MB) are read past the caches: 16384 rows of 2048 with
// an fp32 residual 78 -> 74 us; of less, where the call before has left them there, 16384 rows of 1000
// in bf16 21 -> 25. (The backward, whose registers have no room for both, always does: 106 -> 97 us and
// 26.1 -> 26.4.)
static bool streamed(long rows, int D, int bytes) { return rows * D * bytes > (128L << 20); }
static int size_of(int dtype) { return dtype == 0 ? 2 : 4; }

hipError_t launch_residual_norm(const ResidualNormArgs& args) {
  ResidualNormArgs a = args;
  a.stream_rows = streamed(a.rows, a.D, size_of(a.dtype) + (a.r ? size_of(a.r_dtype) : 0));
  if (a.dtype == 1) return norm_launch<float, float>(a);
  return a.r_dtype == 1 ? norm_launch<bf16, float>(a) : norm_launch<bf16, bf16>(a);
}

hipError_t launch_residual_norm_bwd(const ResidualNormBwdArgs& a) {
  if (a.dtype == 1) return norm_bwd_launch<float, float>(a);
  return a.r_dtype == 1 ? norm_bwd_launch<bf16, float>(a) : norm_bwd_launch<bf16, bf16>(a);
}

}  // namespace gdn2
