// i8_quantize.hip -- rows of f32, bf16 or f16 to int8 with one f32 scale per row
// (gemmq_quantize_i8): s = max|x| / 127, q = round-half-even(x / s).
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

// One workgroup of T threads per row; a thread keeps up to kHeld 16-byte loads of it in
// registers between the two passes (by 512 threads rows of up to 8192 f32 or 16384 bf16 and
// f16 values are read once), and reads what is beyond them again (MORE: there may be such).
constexpr int kHeld = 4;
template <int TYPE, int T, bool MORE>
__global__ __launch_bounds__(T) void quantize_kernel(const void* X, int64_t ldx, bool wide,
                                                     int8_t* Q, int64_t ldq, float* s, int M, int K) {
  constexpr int V = TYPE == GEMMQ_F32 ? 4 : 8, kSpan = T * V;
  __shared__ uint32_t tops[T / 64];
  const int64_t m = blockIdx.y + (int64_t)gridDim.y * blockIdx.z, x0 = m * ldx;
  if (m >= M) return;  // all of the workgroup
  const int t = threadIdx.x;
  uint4 held[kHeld];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = kSpan * i + V * t;
    if (kSpan * i < K) held[i] = load_raw<TYPE>(X, x0 + k, K - k, wide);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (kSpan * i < K) {
      float v[V];
      unpack<TYPE, V>(held[i], v);
#pragma unroll
      for (int e = 0; e < V; ++e) top = max(top, abs_bits(v[e]));
    }
  for (int k = kSpan * kHeld + V * t; MORE && k < K; k += kSpan) {
    float v[V];
    load_values<TYPE, V>(X, x0 + k, K - k, wide, v);
#pragma unroll
    for (int e = 0; e < V; ++e) top = max(top, abs_bits(v[e]));
  }
  top = wave_max(top);
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) top = max(top, tops[w]);
  const float sc = scale_of(top);
  const float inv = 1.0f / sc;
  if (t == 0) s[m] = sc;
  auto store = [&](int k, const float (&v)[V]) {
    uint32_t q[V / 4];
    quantize_values<V>(v, sc, inv, q);
    int8_t* to = Q + m * ldq + k;
    if (k + V <= K) {
#pragma unroll
      for (int w = 0; w < V / 4; ++w) reinterpret_cast<uint32_t*>(to)[w] = q[w];
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (k + e < K) to[e] = (int8_t)(q[e >> 2] >> (8 * (e & 3)));
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (kSpan * i < K) {
      float v[V];
      unpack<TYPE, V>(held[i], v);
      store(kSpan * i + V * t, v);
    }
  for (int k = kSpan * kHeld + V * t; MORE && k < K; k += kSpan) {
    float v[V];
    load_values<TYPE, V>(X, x0 + k, K - k, wide, v);
    store(k, v);
  }
}

template <int TYPE>
void launch_type(const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s, int M, int K,
                 hipStream_t st) {
  const dim3 g = rows_grid(1, M);
  const bool wide = wide_rows(X, ldx, TYPE);
  // 256 threads for a row that is one piece a thread of theirs; of two or three from 768 rows on;
  // of four in f32 where the chip holds all rows' workgroups at once, but not of 512 threads (8
  // and 4 a CU).  Else 512.  (us, 256 / 512 threads:
  //   f32    M = 16    K = 1024 2.8 / 2.8, 2048 3.1 / 2.7, 4096 3.7 / 3.0, 12288 7.0 / 4.7
  //          M = 512   K = 1024 2.8 / 3.2, 2048 3.15 / 3.18, 4096 3.9 / 3.6
  //          M = 1024  K = 2560 4.1 / 4.6, 4096 4.57 / 4.53
  //          M = 2048  K = 1024 3.8 / 5.4, 2560 5.4 / 6.9, 4096 7.3 / 8.5, 5120 11.3 / 11.3
  //          M = 2560  K = 2560 6.9 / 8.2, 4096 11.1 / 10.5
  //   bf16   M = 16    K = 2048 2.8 / 3.2, 4096 3.2 / 2.9, 6144 3.7 / 3.6, 12288 5.3 / 3.9
  //          M = 512   K = 2048 3.1 / 3.8, 4096 3.6 / 3.6, 6144 4.4 / 4.8
  //          M = 1024  K = 4096 4.6 / 4.8, 6144 5.6 / 6.5, 8192 6.9 / 6.8
  //          M = 2048  K = 2048 4.6 / 7.1, 4096 6.3 / 7.1, 6144 8.6 / 9.9, 8192 11.4 / 11.3
  // and f16 as bf16.)
  const int64_t pieces = ceil_div(K, 256 * kValues<TYPE>);
  const bool narrow = pieces == 1 || (pieces <= 3 && M >= 768) ||
                      (TYPE == GEMMQ_F32 && pieces == 4 && M > 1024 && M <= 2048);
  if (narrow)
    quantize_kernel<TYPE, 256, false><<<g, 256, 0, st>>>(X, ldx, wide, Q, ldq, s, M, K);
  else
    quantize_kernel<TYPE, 512, true><<<g, 512, 0, st>>>(X, ldx, wide, Q, ldq, s, M, K);
}

}  // namespace

int launch_quantize(int type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s, int M,
                    int K, hipStream_t st) {
  type == GEMMQ_F32    ? launch_type<GEMMQ_F32>(X, ldx, Q, ldq, s, M, K, st)
  : type == GEMMQ_BF16 ? launch_type<GEMMQ_BF16>(X, ldx, Q, ldq, s, M, K, st)
                       : launch_type<GEMMQ_F16>(X, ldx, Q, ldq, s, M, K, st);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
