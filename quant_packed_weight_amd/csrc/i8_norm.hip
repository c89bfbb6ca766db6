// i8_norm.hip -- the root-mean-square norm between two int8 products (gemmq_rms_i8): the
// residual's addition, the norm's weight and the row quantizer in one pass over the
// rows; and its gradient (gemmq_rms_i8_grad).
//
// The norm of a row is one positive factor rstd: with p = h w, max|p rstd| / 127 is
// rstd max|p| / 127 and the quotients are those of p.  So the integers come from p alone,
// and the sum of squares, taken on the same pass, enters the scale.
#include "i8_block.h"
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

// V values of an f32 vector from element k on, zero from element `end` on
template <int V>
__device__ __forceinline__ void load_vector(const float* w, int k, int end, bool wide,
                                            float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    float four[4];
    load_values<GEMMQ_F32, 4>(w, k + i, end - (k + i), wide, four);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[i + e] = four[e];
  }
}

// the sum over the workgroup of T threads of v[0..N), in every thread and in a fixed
// order; `at`: N * T / 64 doubles of LDS that nothing else uses
template <int T, int N>
__device__ __forceinline__ void sum_all(double (&v)[N], double* at, int t) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], d, 64);
  if ((t & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) at[N * (t >> 6) + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = at[i];
#pragma unroll
  for (int w = 1; w < T / 64; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += at[N * w + i];
}

// One workgroup per row, which is kept in registers (kHeld 16-byte pieces a thread) as
// quantize_kernel keeps it; what is beyond them is read twice.
constexpr int kHeld = 8;

template <int TYPE, int T>
__global__ __launch_bounds__(T) void rms_kernel(RmsArgs a) {
  constexpr int V = kValues<TYPE>, kSpan = T * V;
  __shared__ uint32_t tops[T / 64];
  __shared__ double sums[T / 64];
  const int64_t m = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  if (m >= a.M) return;  // all of the workgroup
  const int t = threadIdx.x, K = a.K;
  const int64_t x0 = m * a.ldx, r0 = m * a.ldr, h0 = m * a.ldh;

  uint4 held[kHeld], add[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = kSpan * i + V * t;
    if (kSpan * i < K) {
      held[i] = load_raw<TYPE>(a.X, x0 + k, K - k, a.wide_x);
      if (a.R) add[i] = load_raw<TYPE>(a.R, r0 + k, K - k, a.wide_r);
    }
  }
  uint32_t top = 0;
  double ss[1] = {0.0};
  // h of 16 bytes, its share of the two statistics taken and H written
  auto take = [&](int k, uint4 x, uint4 r) {
    float v[V], w[V];
    unpack<TYPE, V>(x, v);
    if (a.R) {
      float o[V];
      unpack<TYPE, V>(r, o);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += o[e];
      x = pack<TYPE, V>(v);
      unpack<TYPE, V>(x, v);
    }
    if (a.H) store_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h, x);
    load_vector<V>(a.w, k, K, a.wide_w, w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      top = max(top, abs_bits(v[e] * w[e]));
      ss[0] = fma((double)v[e], (double)v[e], ss[0]);
    }
    return x;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (kSpan * i < K) held[i] = take(kSpan * i + V * t, held[i], add[i]);
  for (int k = kSpan * kHeld + V * t; k < K; k += kSpan) {
    const uint4 x = load_raw<TYPE>(a.X, x0 + k, K - k, a.wide_x);
    take(k, x, a.R ? load_raw<TYPE>(a.R, r0 + k, K - k, a.wide_r) : x);
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if ((t & 63) == 0) tops[t >> 6] = top;
  sum_all<T>(ss, sums, t);
  top = tops[0];
#pragma unroll
  for (int w = 1; w < T / 64; ++w) top = max(top, tops[w]);
  const float sc = scale_of(top);
  const float inv = 1.0f / sc;
  // (a row of zeros has the scale 0 whatever eps is)
  if (t == 0)
    a.s[m] = sc == 0.0f ? 0.0f : (float)((double)sc / sqrt(ss[0] / K + (double)a.eps));

  auto store = [&](int k, uint4 x) {
    float v[V], w[V];
    unpack<TYPE, V>(x, v);
    load_vector<V>(a.w, k, K, a.wide_w, w);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= w[e];
    uint32_t q[V / 4];
    quantize_values<V>(v, sc, inv, q);
    int8_t* to = a.Q + m * a.ldq + k;
    if (k + V <= K) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) reinterpret_cast<uint32_t*>(to)[i] = q[i];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (k + e < K) to[e] = (int8_t)(q[e >> 2] >> (8 * (e & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (kSpan * i < K) store(kSpan * i + V * t, held[i]);
  // what was not kept: h where it was written (by this thread: X or R may be H), else
  // x + r once more
  for (int k = kSpan * kHeld + V * t; k < K; k += kSpan) {
    if (a.H) {
      store(k, load_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h));
      continue;
    }
    uint4 x = load_raw<TYPE>(a.X, x0 + k, K - k, a.wide_x);
    if (a.R) {
      float v[V], o[V];
      unpack<TYPE, V>(x, v);
      load_values<TYPE, V>(a.R, r0 + k, K - k, a.wide_r, o);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] += o[e];
      x = pack<TYPE, V>(v);
    }
    store(k, x);
  }
}

// The gradient, workgroup g of G the rows g, g + G, ...: a row is read once (HELD 16-byte
// pieces a thread of h and of dy; HELD == 0: rows of any width, read twice), and a
// thread's columns are the same in each row, so its sums for dw stay in registers
// (HELD == 0: in the workgroup's row of `part`) and are added up by join_kernel.
template <int TYPE, int T, int HELD, bool DW>
__global__ __launch_bounds__(T) void rms_grad_kernel(RmsGradArgs a) {
  constexpr int V = kValues<TYPE>, kSpan = T * V, kKeep = HELD > 0 ? HELD : 1;
  __shared__ double sums[2][2 * T / 64];
  const int t = threadIdx.x, K = a.K;
  float* part = DW ? a.part + (int64_t)blockIdx.x * a.kp : nullptr;

  float w[kKeep][V], dw[DW ? kKeep : 1][V];
  if constexpr (HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int k = kSpan * i + V * t;
      if (kSpan * i < K) load_vector<V>(a.w, k, K, a.wide_w, w[i]);
      if constexpr (DW) {
#pragma unroll
        for (int e = 0; e < V; ++e) dw[i][e] = 0.0f;
      }
    }
  }
  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const int64_t h0 = m * a.ldh, y0 = m * a.lddy, d0 = m * a.lddh, x0 = m * a.lddx;
    uint4 hr[kKeep], yr[kKeep];
    double s[2] = {0.0, 0.0};  // of h^2 and of d h
    auto take = [&](uint4 hw, uint4 yw, const float(&wv)[V]) {
      float h[V], y[V];
      unpack<TYPE, V>(hw, h);
      unpack<TYPE, V>(yw, y);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        s[0] = fma((double)h[e], (double)h[e], s[0]);
        s[1] = fma((double)(y[e] * wv[e]), (double)h[e], s[1]);
      }
    };
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const int k = kSpan * i + V * t;
        if (kSpan * i < K) {
          hr[i] = load_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h);
          yr[i] = load_raw<TYPE>(a.dY, y0 + k, K - k, a.wide_dy);
        }
      }
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) take(hr[i], yr[i], w[i]);
    } else {
      for (int k = V * t; k < K; k += kSpan) {
        load_vector<V>(a.w, k, K, a.wide_w, w[0]);
        take(load_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h),
             load_raw<TYPE>(a.dY, y0 + k, K - k, a.wide_dy), w[0]);
      }
    }
    // (two sets of LDS: a wave may be a row ahead of one that still reads the sums)
    sum_all<T>(s, sums[turn], t);
    const double r = 1.0 / sqrt(s[0] / K + (double)a.eps);
    const float rstd = (float)r, mean = (float)(s[1] * r / K);
    auto give = [&](int k, uint4 hw, uint4 yw, const float(&wv)[V], float(&dwv)[V]) {
      float h[V], y[V], dx[V];
      unpack<TYPE, V>(hw, h);
      unpack<TYPE, V>(yw, y);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = h[e] * rstd;
        dx[e] = rstd * fmaf(-n, mean, y[e] * wv[e]);
        if constexpr (DW) dwv[e] = fmaf(y[e], n, dwv[e]);
      }
      if (a.dH) {
        float o[V];
        load_values<TYPE, V>(a.dH, d0 + k, K - k, a.wide_dh, o);
#pragma unroll
        for (int e = 0; e < V; ++e) dx[e] += o[e];
      }
      store_raw<TYPE>(a.dX, x0 + k, K - k, a.wide_dx, pack<TYPE, V>(dx));
    };
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) give(kSpan * i + V * t, hr[i], yr[i], w[i], dw[DW ? i : 0]);
    } else {
      for (int k = V * t; k < K; k += kSpan) {
        load_vector<V>(a.w, k, K, a.wide_w, w[0]);
        if constexpr (DW) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            dw[0][e] = m < gridDim.x || k + e >= a.kp ? 0.0f : part[k + e];
        }
        give(k, load_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h),
             load_raw<TYPE>(a.dY, y0 + k, K - k, a.wide_dy), w[0], dw[0]);
        if constexpr (DW) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (k + e < a.kp) part[k + e] = dw[0][e];
        }
      }
    }
  }
  if constexpr (DW && HELD > 0) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int k = kSpan * i + V * t;
#pragma unroll
      for (int e = 0; e < V; e += 4)
        if (k + e < a.kp)  // a multiple of 4
          *reinterpret_cast<float4*>(part + k + e) =
              make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
    }
  }
}

// out[k] = the sum of part[g][k] over g < count, 64 columns a workgroup, its four waves a
// quarter of the rows each
__global__ __launch_bounds__(256) void join_kernel(const float* part, int64_t pitch, int count,
                                                   float* out, int K) {
  __shared__ float sums[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;
  const int each = (count + 3) / 4, end = min(count, each * (wave + 1));
  float s = 0.0f;
  if (k < K) {
#pragma unroll 8
    for (int g = each * wave; g < end; ++g) s += part[g * pitch + k];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && k < K)
    out[k] = (sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]);
}

template <int TYPE, bool DW>
void launch_grad(const RmsGradArgs& a, int groups, hipStream_t st) {
  constexpr int V = kValues<TYPE>;
  if (a.K <= 256 * 2 * V)
    rms_grad_kernel<TYPE, 256, 2, DW><<<groups, 256, 0, st>>>(a);
  else if (a.K <= 256 * 4 * V)
    rms_grad_kernel<TYPE, 256, 4, DW><<<groups, 256, 0, st>>>(a);
  else
    rms_grad_kernel<TYPE, 1024, 0, DW><<<groups, 1024, 0, st>>>(a);
}

}  // namespace

int launch_rms(const RmsArgs& a, hipStream_t st) {
  const dim3 g = rows_grid(1, a.M);
  if (a.type == GEMMQ_F32)
    rms_kernel<GEMMQ_F32, 256><<<g, 256, 0, st>>>(a);
  else if (a.type == GEMMQ_BF16)
    rms_kernel<GEMMQ_BF16, 256><<<g, 256, 0, st>>>(a);
  else
    rms_kernel<GEMMQ_F16, 256><<<g, 256, 0, st>>>(a);
  return 0;
}

int rms_grad_groups(int64_t M) { return (int)(M < 512 ? M : 512); }

int launch_rms_grad(const RmsGradArgs& a, hipStream_t st) {
  const int g = rms_grad_groups(a.M);
  const bool dw = a.part != nullptr;
  if (a.type == GEMMQ_F32)
    dw ? launch_grad<GEMMQ_F32, true>(a, g, st) : launch_grad<GEMMQ_F32, false>(a, g, st);
  else if (a.type == GEMMQ_BF16)
    dw ? launch_grad<GEMMQ_BF16, true>(a, g, st) : launch_grad<GEMMQ_BF16, false>(a, g, st);
  else
    dw ? launch_grad<GEMMQ_F16, true>(a, g, st) : launch_grad<GEMMQ_F16, false>(a, g, st);
  return 0;
}

int launch_join(const float* part, int64_t pitch, int count, float* out, int K, hipStream_t st) {
  join_kernel<<<(uint32_t)ceil_div(K, 64), 256, 0, st>>>(part, pitch, count, out, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
