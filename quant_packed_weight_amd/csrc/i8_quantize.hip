// i8_quantize.hip -- rows of f32, bf16 or f16 to int8 with one f32 scale per row
// (gemmq_quantize_i8): s = max|x| / 127, q = round-half-even(x / s).
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

// One workgroup per row; a thread keeps up to kHeld 16-byte loads of it in
// registers between the two passes (rows of up to 8192 f32 or 16384 bf16 and f16
// values are read once), and reads what is beyond them again.
constexpr int kHeld = 8;

template <int TYPE>
__global__ __launch_bounds__(256) void quantize_kernel(const void* X, int64_t ldx, bool wide,
                                                       int8_t* Q, int64_t ldq, float* s, int M, int K) {
  constexpr int V = TYPE == GEMMQ_F32 ? 4 : 8, kSpan = 256 * V;
  __shared__ uint32_t tops[4];
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
  for (int k = kSpan * kHeld + V * t; k < K; k += kSpan) {
    float v[V];
    load_values<TYPE, V>(X, x0 + k, K - k, wide, v);
#pragma unroll
    for (int e = 0; e < V; ++e) top = max(top, abs_bits(v[e]));
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if ((t & 63) == 0) tops[t >> 6] = top;
  __syncthreads();
  const float sc = scale_of(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
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
  for (int k = kSpan * kHeld + V * t; k < K; k += kSpan) {
    float v[V];
    load_values<TYPE, V>(X, x0 + k, K - k, wide, v);
    store(k, v);
  }
}

}  // namespace

int launch_quantize(int type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s, int M,
                    int K, hipStream_t st) {
  const dim3 g = rows_grid(1, M);
  const bool wide = wide_rows(X, ldx, type);
  if (type == GEMMQ_F32)
    quantize_kernel<GEMMQ_F32><<<g, 256, 0, st>>>(X, ldx, wide, Q, ldq, s, M, K);
  else if (type == GEMMQ_BF16)
    quantize_kernel<GEMMQ_BF16><<<g, 256, 0, st>>>(X, ldx, wide, Q, ldq, s, M, K);
  else
    quantize_kernel<GEMMQ_F16><<<g, 256, 0, st>>>(X, ldx, wide, Q, ldq, s, M, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
