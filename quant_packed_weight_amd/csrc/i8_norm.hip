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

// Of a row, h and what is read to make it, and in the gradient h (which the forward pass left
// long ago) and dx, are accessed as streams (ONCE) that the L2 need not keep; dy and dh come
// from the calls just before.  Out of memory, in bf16, that takes the norm of 2048 x 4096 from
// 17.6 to 14.8 us and of 8192 x 4096 from 53 to 46, the gradient from 21.6 to 20.8 and from 57.5
// to 54.6 (dy and dh as streams too 52.8; but 18 instead of 16 where they are in the caches).
// In a decoder block whose products follow at once there is no difference either way.

// a thread's 16 bytes of a piece of SPAN values from element `first` of a row on (SPAN 0: not
// asked whether all of it is there)
template <int TYPE, int SPAN, bool ONCE>
__device__ __forceinline__ uint4 load_piece(const void* p, int64_t row, int first, int t, int K,
                                            bool wide) {
  constexpr int V = kValues<TYPE>;
  const int k = first + V * t;
  if (SPAN > 0 && wide && first + SPAN <= K)  // the same way in all lanes
    return load_raw<TYPE, ONCE>(p, row + k, V, true);
  return load_raw<TYPE, ONCE>(p, row + k, K - k, wide);
}
template <int TYPE, int SPAN, bool ONCE>
__device__ __forceinline__ void store_piece(void* p, int64_t row, int first, int t, int K,
                                            bool wide, uint4 w) {
  constexpr int V = kValues<TYPE>;
  const int k = first + V * t;
  if (SPAN > 0 && wide && first + SPAN <= K)
    store_raw<TYPE, ONCE>(p, row + k, V, true, w);
  else
    store_raw<TYPE, ONCE>(p, row + k, K - k, wide, w);
}

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

// The norm, workgroup g of G the rows g, g + G, ...: a row is read once (HELD 16-byte pieces
// a thread), the next one's loads under way while it is worked on, and the weights stay in
// registers.  HELD == 0: rows of any width, read twice.
template <int TYPE, int T, int HELD>
__global__ __launch_bounds__(T) void rms_kernel(RmsArgs a) {
  constexpr int V = kValues<TYPE>, kSpan = T * V, kKeep = HELD > 0 ? HELD : 1;
  __shared__ uint32_t tops[2][T / 64];
  __shared__ double sums[2][T / 64];
  const int t = threadIdx.x, K = a.K;
  float w[kKeep][V];
  uint4 x[kKeep], r[kKeep];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (kSpan * i < K) {
        x[i] = load_piece<TYPE, kSpan, true>(a.X, m * a.ldx, kSpan * i, t, K, a.wide_x);
        if (a.R) r[i] = load_piece<TYPE, kSpan, true>(a.R, m * a.ldr, kSpan * i, t, K, a.wide_r);
      }
    }
  };
  // h of 16 bytes
  auto add = [&](uint4 xw, uint4 rw) {
    if (!a.R) return xw;
    float v[V], o[V];
    unpack<TYPE, V>(xw, v);
    unpack<TYPE, V>(rw, o);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += o[e];
    return pack<TYPE, V>(v);
  };
  load(blockIdx.x);
#pragma unroll
  for (int i = 0; i < HELD; ++i)
    if (kSpan * i < K) load_vector<V>(a.w, kSpan * i + V * t, K, a.wide_w, w[i]);

  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    uint32_t top = 0;
    double ss[1] = {0.0};
    // the share of 16 bytes of h in the two statistics, and H written
    auto take = [&](int first, uint4 h, const float(&wv)[V]) {
      if (a.H) store_piece<TYPE, kSpan, (HELD > 0)>(a.H, m * a.ldh, first, t, K, a.wide_h, h);
      float v[V];
      unpack<TYPE, V>(h, v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        top = max(top, abs_bits(v[e] * wv[e]));
        ss[0] = fma((double)v[e], (double)v[e], ss[0]);
      }
    };
    uint4 held[kKeep];
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) held[i] = add(x[i], r[i]);
      if (m + gridDim.x < a.M) load(m + gridDim.x);
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) take(kSpan * i, held[i], w[i]);
    } else {
      for (int k = V * t; k < K; k += kSpan) {
        const uint4 xw = load_raw<TYPE>(a.X, m * a.ldx + k, K - k, a.wide_x);
        const uint4 h = add(xw, a.R ? load_raw<TYPE>(a.R, m * a.ldr + k, K - k, a.wide_r) : xw);
        load_vector<V>(a.w, k, K, a.wide_w, w[0]);
        take(k - V * t, h, w[0]);
      }
    }
    top = wave_max(top);
    if ((t & 63) == 0) tops[turn][t >> 6] = top;
    // (two sets of LDS: a wave may be a row ahead of one that still reads them)
    sum_all<T>(ss, sums[turn], t);
    top = tops[turn][0];
#pragma unroll
    for (int i = 1; i < T / 64; ++i) top = max(top, tops[turn][i]);
    const float sc = scale_of(top);
    const float inv = 1.0f / sc;
    // (a row of zeros has the scale 0 whatever eps is)
    if (t == 0)
      a.s[m] = sc == 0.0f ? 0.0f : (float)((double)sc / sqrt(ss[0] / K + (double)a.eps));
    auto store = [&](int k, uint4 h, const float(&wv)[V]) {
      float v[V];
      unpack<TYPE, V>(h, v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] *= wv[e];
      uint32_t q[V / 4];
      quantize_values<V>(v, sc, inv, q);
      int8_t* to = a.Q + m * a.ldq + k;
      if (k + V <= K) {
        if constexpr (V == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
        else
          *reinterpret_cast<uint32_t*>(to) = q[0];
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (k + e < K) to[e] = (int8_t)(q[e >> 2] >> (8 * (e & 3)));
      }
    };
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) store(kSpan * i + V * t, held[i], w[i]);
    } else {
      // h where it was written (by this thread: X or R may be H), else x + r once more
      for (int k = V * t; k < K; k += kSpan) {
        load_vector<V>(a.w, k, K, a.wide_w, w[0]);
        if (a.H) {
          store(k, load_raw<TYPE>(a.H, m * a.ldh + k, K - k, a.wide_h), w[0]);
          continue;
        }
        const uint4 xw = load_raw<TYPE>(a.X, m * a.ldx + k, K - k, a.wide_x);
        store(k, add(xw, a.R ? load_raw<TYPE>(a.R, m * a.ldr + k, K - k, a.wide_r) : xw), w[0]);
      }
    }
  }
}

// The gradient, workgroup g of G the rows g, g + G, ...: a row is read once (HELD 16-byte
// pieces a thread of h and of dy; HELD == 0: rows of any width, read twice), and a
// thread's columns are the same in each row, so its sums for dw stay in registers
// (HELD == 0: in the workgroup's row of `part`) and are added up by join_kernel.
// BARE: eps is 0.  A row of zeros then has no gradient (the forward pass has the scale 0 for it),
// and of a row of subnormal values rstd passes f32: its h is scaled up by 2^64, which is exact,
// rstd down, and dx up again.  (With an eps that would cost 2048 x 4096 in bf16 19.1 instead of
// 18.8 us.)
template <int TYPE, int T, int HELD, bool DW, bool BARE>
__global__ __launch_bounds__(T) void rms_grad_kernel(RmsGradArgs a) {
  constexpr int V = kValues<TYPE>, kSpan = T * V, kKeep = HELD > 0 ? HELD : 1;
  constexpr int kPiece = HELD < 4 ? kSpan : 0;  // (of four, two ways to each leave registers short)
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
  // the next row's pieces
  uint4 hn[kKeep], yn[kKeep], dn[kKeep];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      if (kSpan * i < K) {
        hn[i] = load_piece<TYPE, kPiece, true>(a.H, m * a.ldh, kSpan * i, t, K, a.wide_h);
        yn[i] = load_piece<TYPE, kPiece, false>(a.dY, m * a.lddy, kSpan * i, t, K, a.wide_dy);
        if (a.dH)
          dn[i] = load_piece<TYPE, kPiece, false>(a.dH, m * a.lddh, kSpan * i, t, K, a.wide_dh);
      }
    }
  };
  load(blockIdx.x);
  int turn = 0;
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const int64_t h0 = m * a.ldh, y0 = m * a.lddy, d0 = m * a.lddh, x0 = m * a.lddx;
    uint4 hr[kKeep], yr[kKeep], dr[kKeep];
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
      for (int i = 0; i < HELD; ++i) hr[i] = hn[i], yr[i] = yn[i], dr[i] = dn[i];
      if (m + gridDim.x < a.M) load(m + gridDim.x);
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
    double r = 1.0 / sqrt(s[0] / K + (double)a.eps);
    if (BARE && r > 0x1p500) r = 0.0;
    const bool far = BARE && r > 0x1p126;
    const float up = far ? 0x1p64f : 1.0f;
    const float rstd = (float)(far ? r * 0x1p-64 : r), mean = (float)(s[1] * r / K);
    auto give = [&](int first, uint4 hw, uint4 yw, uint4 dw4, const float(&wv)[V], float(&dwv)[V]) {
      float h[V], y[V], dx[V];
      unpack<TYPE, V>(hw, h);
      unpack<TYPE, V>(yw, y);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float n = h[e] * up * rstd;
        dx[e] = rstd * fmaf(-n, mean, y[e] * wv[e]) * up;
        if constexpr (DW) dwv[e] = fmaf(y[e], n, dwv[e]);
      }
      if (a.dH) {
        float o[V];
        unpack<TYPE, V>(dw4, o);
#pragma unroll
        for (int e = 0; e < V; ++e) dx[e] += o[e];
      }
      store_piece<TYPE, kPiece, true>(a.dX, x0, first, t, K, a.wide_dx, pack<TYPE, V>(dx));
    };
    if constexpr (HELD > 0) {
#pragma unroll
      for (int i = 0; i < HELD; ++i)
        if (kSpan * i < K) give(kSpan * i, hr[i], yr[i], dr[i], w[i], dw[DW ? i : 0]);
    } else {
      for (int k = V * t; k < K; k += kSpan) {
        load_vector<V>(a.w, k, K, a.wide_w, w[0]);
        if constexpr (DW) {
#pragma unroll
          for (int e = 0; e < V; ++e)
            dw[0][e] = m < gridDim.x || k + e >= a.kp ? 0.0f : part[k + e];
        }
        const uint4 h = load_raw<TYPE>(a.H, h0 + k, K - k, a.wide_h);
        give(k - V * t, h, load_raw<TYPE>(a.dY, y0 + k, K - k, a.wide_dy),
             a.dH ? load_raw<TYPE>(a.dH, d0 + k, K - k, a.wide_dh) : h, w[0], dw[0]);
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
      for (int e = 0; e < V; e += 4) {
        if (k + e >= a.kp) continue;
        if (a.wide_part) {
          *reinterpret_cast<float4*>(part + k + e) =
              make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
        } else {
#pragma unroll
          for (int f = e; f < e + 4; ++f)
            if (k + f < a.kp) part[k + f] = dw[i][f];
        }
      }
    }
  }
}

// out[k] = the sum of part[g][k] over g < count: 64 columns a workgroup, its waves a
// sixteenth of the rows each
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(Join a, Join b, int64_t pitch,
                                                               int count, int K) {
  __shared__ float sums[kJoinWaves][64];
  const float* part = blockIdx.y ? b.part : a.part;
  float* out = blockIdx.y ? b.out : a.out;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane;
  const int each = (count + kJoinWaves - 1) / kJoinWaves, end = min(count, each * (wave + 1));
  float s = 0.0f;
  if (k < K) {
#pragma unroll 8
    for (int g = each * wave; g < end; ++g) s += part[g * pitch + k];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave > 0 || k >= K) return;
#pragma unroll
  for (int w = 1; w < kJoinWaves; ++w) s += sums[w][lane];
  out[k] = s;
}

// Threads a row (us, out of memory): up to 4096 16-bit values 256, of more 512 (512 / 256: 1024 x
// 5120 in bf16 13.2 / 15.8, 2048 x 4096 in f32 21 / 31), of f32 beyond 4096 1024 (1024 x 8192 26.9,
// by 512 29.5); of more than 16384 values it is read twice (2048 x 12288 in f32 held 72, read
// twice 90; 512 x 20480 in bf16 32 / 26).  Rows in flight: four waves a SIMD, whatever that is in
// workgroups (half / that / twice: 2048 x 4096 in bf16 18.2 / 14.8 / 17.3; that / twice: 1024 x
// 8192 in bf16 14.7 / 17.5, 2048 x 4096 in f32 22.1 / 23.7, 1024 x 8192 in f32 22.7 / 24.4).
constexpr int kRmsThreads = 1024 * 256;

// In the gradient a row's thread holds three times as much: f32 beyond 4096 by 1024 threads (us,
// 1024 / 512: 1024 x 8192 35.4 / 42.6, 4096 x 8192 109 / 143), and of more than 8192 f32 values it
// is read twice (2048 x 12288 155, by 1024 threads at once 158; 680 x 12288 61 / 73).
template <int TYPE, bool DW, bool BARE>
void launch_grad(const RmsGradArgs& a, int groups, hipStream_t st) {
  constexpr int V = kValues<TYPE>;
  if (a.K <= 256 * 2 * V)
    rms_grad_kernel<TYPE, 256, 2, DW, BARE><<<groups, 256, 0, st>>>(a);
  else if (a.K <= 512 * 2 * V)
    rms_grad_kernel<TYPE, 512, 2, DW, BARE><<<groups, 512, 0, st>>>(a);
  else if (a.K > (TYPE == GEMMQ_F32 ? 1024 * 2 * V : 512 * 4 * V))
    rms_grad_kernel<TYPE, 1024, 0, DW, BARE><<<groups, 1024, 0, st>>>(a);
  else if constexpr (TYPE == GEMMQ_F32)
    rms_grad_kernel<TYPE, 1024, 2, DW, BARE><<<groups, 1024, 0, st>>>(a);
  else
    rms_grad_kernel<TYPE, 512, 4, DW, BARE><<<groups, 512, 0, st>>>(a);
}

template <int TYPE>
void launch_grad(const RmsGradArgs& a, int groups, hipStream_t st) {
  const bool dw = a.part != nullptr;
  if (a.eps == 0.0f)
    dw ? launch_grad<TYPE, true, true>(a, groups, st) : launch_grad<TYPE, false, true>(a, groups, st);
  else
    dw ? launch_grad<TYPE, true, false>(a, groups, st) : launch_grad<TYPE, false, false>(a, groups, st);
}

template <int TYPE, int T, int HELD>
void launch_rows(const RmsArgs& a, hipStream_t st) {
  const int most = kRmsThreads / T;
  rms_kernel<TYPE, T, HELD><<<a.M < most ? a.M : most, T, 0, st>>>(a);
}

template <int TYPE>
void launch_type(const RmsArgs& a, hipStream_t st) {
  constexpr int V = kValues<TYPE>;
  if (a.K <= 256 * 2 * V)
    launch_rows<TYPE, 256, 2>(a, st);
  else if (a.K <= 512 * 2 * V)
    launch_rows<TYPE, 512, 2>(a, st);
  else if (a.K > 16384)
    launch_rows<TYPE, 1024, 0>(a, st);
  else if constexpr (TYPE != GEMMQ_F32)
    launch_rows<TYPE, 512, 4>(a, st);
  else if (a.K <= 1024 * 2 * V)
    launch_rows<TYPE, 1024, 2>(a, st);
  else
    launch_rows<TYPE, 1024, 4>(a, st);
}

}  // namespace

int launch_rms(const RmsArgs& a, hipStream_t st) {
  a.type == GEMMQ_F32    ? launch_type<GEMMQ_F32>(a, st)
  : a.type == GEMMQ_BF16 ? launch_type<GEMMQ_BF16>(a, st)
                         : launch_type<GEMMQ_F16>(a, st);
  return 0;
}

// As many workgroups as the CUs hold: two each, of rows beyond 4096 one, whose threads keep
// twice as much (us with 512 and 256 workgroups: bf16, 2048 x 4096 17.0 / 19.6, 1024 x 8192 24.8
// / 19.6, 680 x 12288 27.8 / 22.6; f32, 2048 x 4096 27.9 / 31.5, 1024 x 8192 37.8 / 33.9).  Without
// partial sums two are never slower by more than 6% (f32, 2048 x 4096 23.9 / 28.7).
// A few short rows go through one workgroup, whose sums are dw itself: a launch less.  A call in
// bf16 that way is 8.0 us of 2 x 4096, 8.5 of 4 x 4096, 10.0 of 2 x 12288 and 16.1 of 4 x 12288;
// one that joins the sums of five workgroups 12.5 at any of these widths.
int rms_grad_groups(int64_t M, int64_t K) {
  const int64_t most = M <= 4 && M * K <= 24576 ? 1 : K <= 4096 ? 512 : 256;
  return (int)(M < most ? M : most);
}

int launch_rms_grad(const RmsGradArgs& a, hipStream_t st) {
  const int g = a.part ? rms_grad_groups(a.M, a.K) : a.M < 512 ? a.M : 512;
  a.type == GEMMQ_F32    ? launch_grad<GEMMQ_F32>(a, g, st)
  : a.type == GEMMQ_BF16 ? launch_grad<GEMMQ_BF16>(a, g, st)
                         : launch_grad<GEMMQ_F16>(a, g, st);
  return 0;
}

int launch_join(Join a, Join b, int64_t pitch, int count, int K, hipStream_t st) {
  if (!a.out) a = b, b.out = nullptr;
  const dim3 grid((uint32_t)ceil_div(K, 64), b.out ? 2 : 1);
  join_kernel<<<grid, 64 * kJoinWaves, 0, st>>>(a, b, pitch, count, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
