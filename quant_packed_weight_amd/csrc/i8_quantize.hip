// i8_quantize.hip -- rows of f32, bf16 or f16 to int8 with one f32 scale per row
// (gemmq_quantize_i8): s = max|x| / 127, q = round-half-even(x / s).
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

// |x| as an unsigned integer: ordered as the values, infinity above every finite
// one and NaN above infinity, so that the maximum shows either.
__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}

// One workgroup per row, two passes over it (the second from cache).
template <int TYPE>
__global__ __launch_bounds__(256) void quantize_kernel(const void* X, int64_t ldx, int8_t* Q,
                                                       int64_t ldq, float* s, int K) {
  __shared__ uint32_t top[4];
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  const int64_t x0 = m * ldx;
  uint32_t a = 0;
  for (int k = t; k < K; k += 256) a = max(a, abs_bits(load_as_f32(X, x0 + k, TYPE)));
  for (int d = 1; d < 64; d *= 2) a = max(a, (uint32_t)__shfl_xor((int)a, d, 64));
  if ((t & 63) == 0) top[t >> 6] = a;
  __syncthreads();
  a = max(max(top[0], top[1]), max(top[2], top[3]));
  const bool finite = a < 0x7f800000u;
  const float d = __builtin_bit_cast(float, a) / 127.0f;
  if (t == 0) s[m] = finite ? d : __builtin_nanf("");
  const bool live = finite && d > 0.0f;
  for (int k = t; k < K; k += 256) {
    const float q = live ? rintf(load_as_f32(X, x0 + k, TYPE) / d) : 0.0f;
    Q[m * ldq + k] = (int8_t)fminf(fmaxf(q, -127.0f), 127.0f);
  }
}

}  // namespace

int launch_quantize(int type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s, int M,
                    int K, hipStream_t st) {
  const dim3 g((uint32_t)M);
  if (type == GEMMQ_F32)
    quantize_kernel<GEMMQ_F32><<<g, 256, 0, st>>>(X, ldx, Q, ldq, s, K);
  else if (type == GEMMQ_BF16)
    quantize_kernel<GEMMQ_BF16><<<g, 256, 0, st>>>(X, ldx, Q, ldq, s, K);
  else
    quantize_kernel<GEMMQ_F16><<<g, 256, 0, st>>>(X, ldx, Q, ldq, s, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
