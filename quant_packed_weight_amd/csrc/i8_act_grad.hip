// i8_act_grad.hip -- the gradients with respect to what is before the activation of a
// linear layer or of a gated pair, and to the biases (gemmq_act_grad).
//
// A stream: two or three matrices in, one or two out.  A wave takes 64 16-byte pieces of
// a row (512 columns of 16 bits, 256 of f32) and every fourth row of its workgroup's range,
// so the sums over rows stay in its lanes; the workgroup's four waves add theirs in LDS
// and the ranges' are added up by launch_join.  (One range's are the sums.)
// All accesses are a stream's, which the L2 need not keep: of 2048 x 12288 in bf16, a pair, 46.2
// -> 42 us, of 8192 x 12288 186 -> 170 (5.9 TB/s), and with the products that take the gradients
// on (2048 and 8192 rows) 488 -> 483 and 1730 -> 1724.
#include "i8_act.h"

namespace gemmq {
namespace i8 {
namespace {

constexpr int kWaves = 4;

template <int TYPE, bool PAIR, bool SUMS>
__global__ __launch_bounds__(64 * kWaves) void act_grad_kernel(ActGradArgs a) {
  constexpr int V = kValues<TYPE>, OUT = PAIR ? 2 : 1;
  __shared__ float sums[SUMS ? kWaves * OUT * 64 * V : 1];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t n = ((int64_t)blockIdx.x * 64 + lane) * V;
  const Act act = act_of(a.act);
  const int left = (int)min((int64_t)V, a.N - n);  // none or fewer: nothing is accessed
  float total[OUT][V];
#pragma unroll
  for (int o = 0; o < OUT; ++o)
#pragma unroll
    for (int e = 0; e < V; ++e) total[o][e] = 0.0f;

  const int64_t group = blockIdx.y;
  const int64_t begin = group * a.M / a.groups, end = (group + 1) * a.M / a.groups;
  for (int64_t m = begin + wave; m < end; m += kWaves) {
    float z[V], y[V], u[V], dz[V], du[V];
    const uint4 zr = load_raw<TYPE, true>(a.Z.p, m * a.Z.ld + n, left, a.Z.lines);
    const uint4 yr = load_raw<TYPE, true>(a.dY.p, m * a.dY.ld + n, left, a.dY.lines);
    if constexpr (PAIR)
      unpack<TYPE, V>(load_raw<TYPE, true>(a.U.p, m * a.U.ld + n, left, a.U.lines), u);
    unpack<TYPE, V>(zr, z);
    unpack<TYPE, V>(yr, y);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float value, slope;
      activate_slope(act, z[e], value, slope);
      dz[e] = y[e] * slope;
      if constexpr (PAIR) {
        dz[e] *= u[e];
        du[e] = y[e] * value;
      }
      if constexpr (SUMS) {
        total[0][e] += dz[e];
        if constexpr (PAIR) total[1][e] += du[e];
      }
    }
    store_raw<TYPE, true>(a.dZ.p, m * a.dZ.ld + n, left, a.dZ.lines, pack<TYPE, V>(dz));
    if constexpr (PAIR)
      store_raw<TYPE, true>(a.dU.p, m * a.dU.ld + n, left, a.dU.lines, pack<TYPE, V>(du));
  }
  if constexpr (SUMS) {
#pragma unroll
    for (int o = 0; o < OUT; ++o)
#pragma unroll
      for (int e = 0; e < V; ++e) sums[((wave * OUT + o) * V + e) * 64 + lane] = total[o][e];
    __syncthreads();
    // column 64 V blockIdx.x + c, of lane c / V and value c mod V
    for (int i = t; i < OUT * 64 * V; i += 64 * kWaves) {
      const int o = i / (64 * V), c = i % (64 * V), at = c % V * 64 + c / V;
      const int64_t col = (int64_t)blockIdx.x * 64 * V + c;
      if (col >= a.N) continue;
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += sums[(w * OUT + o) * V * 64 + at];
      if (a.sums[o]) a.sums[o][group * a.np + col] = s;
    }
  }
}

template <int TYPE>
int launch_type(const ActGradArgs& a, hipStream_t st) {
  const int64_t strips = ceil_div(a.N, 64 * kValues<TYPE>);
  const dim3 grid((uint32_t)strips, (uint32_t)a.groups);
  const bool pair = a.U.p != nullptr;
  if (a.sums[0] || a.sums[1])
    pair ? act_grad_kernel<TYPE, true, true><<<grid, 64 * kWaves, 0, st>>>(a)
         : act_grad_kernel<TYPE, false, true><<<grid, 64 * kWaves, 0, st>>>(a);
  else
    pair ? act_grad_kernel<TYPE, true, false><<<grid, 64 * kWaves, 0, st>>>(a)
         : act_grad_kernel<TYPE, false, false><<<grid, 64 * kWaves, 0, st>>>(a);
  return 0;
}

// ranges of rows: enough workgroups to fill the chip several times, but no more than a quarter
// of the rows (rounded up): a row for each wave
int ranges(int type, int64_t M, int64_t N, int64_t most) {
  const int64_t strips = ceil_div(N, type == GEMMQ_F32 ? 256 : 512);
  int64_t g = ceil_div(most, strips);
  if (g > ceil_div(M, 4)) g = ceil_div(M, 4);
  return (int)(g < 1 ? 1 : g > 32768 ? 32768 : g);
}

}  // namespace

// Up to 16 rows (four a wave) go through one workgroup for each strip of columns, whose sums
// are the gradients of the biases themselves: a launch less (N = 4096 in bf16, a call with a
// bias's gradient 7.7 us of 16 rows, 12.2 of 17; of a gated pair with both 9.1 and 13.6).
int act_grad_groups(int type, int64_t M, int64_t N) {
  return M <= 16 ? 1 : ranges(type, M, N, 1024);
}

int launch_act_grad(ActGradArgs a, hipStream_t st) {
  a.groups = a.sums[0] || a.sums[1] ? act_grad_groups(a.type, a.M, a.N)
                                    : ranges(a.type, a.M, a.N, 16384);
  return a.type == GEMMQ_F32    ? launch_type<GEMMQ_F32>(a, st)
         : a.type == GEMMQ_BF16 ? launch_type<GEMMQ_BF16>(a, st)
                                : launch_type<GEMMQ_F16>(a, st);
}

}  // namespace i8
}  // namespace gemmq
