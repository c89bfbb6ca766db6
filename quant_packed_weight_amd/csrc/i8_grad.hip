// i8_grad.hip -- the product that both gradients need, acc[m, k] = sum_n
// A[m, n] W[n, k]: int8 weights, exact in bf16, against a factor A given as one
// to three bf16 matrices whose sum it is; and the kernels before and after it.
//
// W is read as it lies, rows of N along the reduction, so its fragments are
// transposed on the way from LDS to registers.  W^T is the MFMA's row operand: a
// lane ends with one token and four consecutive k per register quad.
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kRed = 64;   // n per step: rows of 64 bytes of W's tile, 128 bytes of A's
constexpr int kBK = 128;   // k per workgroup

__device__ __forceinline__ v16f mfma_bf16(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <int BM, int WK, int WM>
__global__ __launch_bounds__(64 * WK * WM) void grad_kernel(GradArgs a, uint32_t ktiles,
                                                            uint32_t mtiles) {
  constexpr int NW = WK * WM;
  constexpr int TK = kBK / WK / 32, TM = BM / WM / 32;
  constexpr int kStageBytes = kRed * kBK + BM * 2 * kRed;
  static_assert(kRed % (8 * NW) == 0 && BM % (8 * NW) == 0, "whole loads per wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStageBytes];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wk = wave % WK, wm = wave / WK;
  uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(id % mtiles) * BM;
  id /= mtiles;
  const int k0 = (int)(id % ktiles) * kBK, split = (int)(id / ktiles);

  // this split's share of the steps; a step has one load of W and A per plane
  const int steps = (a.N + kRed - 1) / kRed;
  const int per = steps / a.splits, more = steps % a.splits;
  const int first = split * per + min(split, more), count = per + (split < more ? 1 : 0);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int r8 = lane >> 3, chunk = 16 * ((lane & 7) ^ r8);
  // chunks of W past column K repeat the last one: their columns are dropped
  const int col = min(k0 + chunk, (a.K - 1) / 16 * 16);
  const int mvalid = (int)min((int64_t)BM, a.M - m0);
  const uint32_t arow = (uint32_t)(2 * a.pitch);

  auto issue = [&](int it, uint32_t dst) {
    const int step = first + it / a.planes, plane = it % a.planes;
    const int64_t n = (int64_t)step * kRed;
    const int nvalid = (int)min((int64_t)kRed, a.N - n);
    const rsrc_t rw = gk::make_rsrc(a.W + n * a.ldw, (uint32_t)(nvalid * a.ldw));
    // rows of W past the last one repeat it: the factor is zero there
#pragma unroll
    for (int j = 0; j < kRed / 8 / NW; ++j) {
      const int r = min(8 * (wave + NW * j) + r8, nvalid - 1);
      gk::dma16(rw, (uint32_t)(r * a.ldw) + col, 0, dst + 1024 * (wave + NW * j));
    }
    const rsrc_t ra = gk::make_rsrc(a.P + ((int64_t)plane * a.M + m0) * a.pitch,
                                    (uint32_t)(mvalid * (int64_t)arow));
#pragma unroll
    for (int j = 0; j < BM / 8 / NW; ++j) {
      const int r = min(8 * (wave + NW * j) + r8, mvalid - 1);
      gk::dma16(ra, r * arow + (uint32_t)(2 * n) + chunk, 0,
                dst + kRed * kBK + 1024 * (wave + NW * j));
    }
  };

  v16f acc[TK][TM];
#pragma unroll
  for (int i = 0; i < TK; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  const int its = count * a.planes;
  if (its > 0) issue(0, lds0);
  for (int it = 0; it < its; ++it) {
    const uint8_t* cw = lds + (it & 1) * kStageBytes;
    const uint8_t* ca = cw + kRed * kBK;
    gk::wait_vm<0>();
    gk::lds_barrier();
    if (it + 1 < its) issue(it + 1, lds0 + ((it + 1) & 1) * kStageBytes);
#pragma unroll
    for (int q = 0; q < kRed / 16; ++q) {
      v8bf wf[TK], af[TM];
#pragma unroll
      for (int i = 0; i < TK; ++i) {
        const int k = (wk * TK + i) * 32 + (lane & 31);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int n = 16 * q + 8 * (lane >> 5) + e;
          wf[i][e] = (__bf16)(float)(int8_t)cw[n * kBK + 16 * ((k >> 4) ^ (n & 7)) + (k & 15)];
        }
      }
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int m = (wm * TM + j) * 32 + (lane & 31), c = 2 * q + (lane >> 5);
        af[j] = *reinterpret_cast<const v8bf*>(ca + m * 128 + 16 * (c ^ (m & 7)));
      }
#pragma unroll
      for (int i = 0; i < TK; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = mfma_bf16(wf[i], af[j], acc[i][j]);
    }
  }

  const int h = lane >> 5;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + (wm * TM + j) * 32 + (lane & 31);
    if (m >= a.M) continue;
    float* out = a.acc + ((int64_t)split * a.M + m) * a.kp;
#pragma unroll
    for (int i = 0; i < TK; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int k = k0 + (wk * TK + i) * 32 + 8 * g + 4 * h;
        if (k >= a.kp) continue;
        float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                               acc[i][j][4 * g + 3]);
        float4* p = reinterpret_cast<float4*>(out + k);
        if (a.add) {
          const float4 o = *p;
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        *p = v;
      }
  }
}

// A[m, n] = dY[m, n] * sw[n] as `planes` bf16 matrices, zero from column N to
// the pitch.  One thread per four columns.
__global__ __launch_bounds__(256) void planes_kernel(int type, const void* dY, int64_t lddy,
                                                     const float* sw, uint16_t* P, int64_t pitch,
                                                     int planes, int M, int N) {
  const int64_t q = pitch / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / q;
  if (m >= M) return;
  const int64_t n = 4 * (i % q);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = n + e < N ? load_as_f32(dY, m * lddy + n + e, type) * sw[n + e] : 0.0f;
  for (int p = 0; p < planes; ++p) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = bf16_part(v[e], p + 1 == planes);
    *reinterpret_cast<uint2*>(P + ((int64_t)p * M + m) * pitch + n) =
        make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  }
}

__global__ __launch_bounds__(256) void finish_kernel(const float* acc, int64_t kp, int splits,
                                                     const float* g, const int64_t* target,
                                                     int64_t nvocab, int type, void* dX,
                                                     int64_t lddx, int M, int K) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / K;
  if (m >= M) return;
  const int64_t k = i % K;
  float v = 0.0f;
  for (int s = 0; s < splits; ++s) v += acc[((int64_t)s * M + m) * kp + k];
  if (g) v *= g[m];
  if (target) {
    const int64_t tg = target[m];
    v = tg < 0 ? 0.0f : tg >= nvocab ? __builtin_nanf("") : v;
  }
  store_as(dX, m * lddx + k, type, v);
}

constexpr int64_t kMaxGrid = 0x7fffffff;
int pick_bm(int M) { return M <= 32 ? 32 : 128; }

}  // namespace

int grad_splits(int M, int N, int K, int) {
  const int64_t tiles = ceil_div(M, pick_bm(M)) * ceil_div(K, kBK);
  const int64_t steps = ceil_div(N, kRed);
  int64_t s = ceil_div(512, tiles);
  if (s > steps / 4) s = steps / 4;
  return s < 1 ? 1 : (int)s;
}

bool grad_fits(int M, int K, int splits) {
  return ceil_div(M, pick_bm(M)) * ceil_div(K, kBK) * splits <= kMaxGrid &&
         ceil_div((int64_t)M * K, 256) <= kMaxGrid;
}

int launch_grad(const GradArgs& a, hipStream_t st) {
  const int bm = pick_bm(a.M);
  const int64_t mt = ceil_div(a.M, bm), kt = ceil_div(a.K, kBK), n = mt * kt * a.splits;
  if (n > kMaxGrid) return -1;
  if (bm == 32)
    grad_kernel<32, 4, 1><<<(uint32_t)n, 256, 0, st>>>(a, (uint32_t)kt, (uint32_t)mt);
  else
    grad_kernel<128, 2, 2><<<(uint32_t)n, 256, 0, st>>>(a, (uint32_t)kt, (uint32_t)mt);
  return 0;
}

int launch_planes(int type, const void* dY, int64_t lddy, const float* sw, uint16_t* P,
                  int64_t pitch, int planes, int M, int N, hipStream_t st) {
  const int64_t n = ceil_div(M * (pitch / 4), 256);
  if (n > kMaxGrid) return -1;
  planes_kernel<<<(uint32_t)n, 256, 0, st>>>(type, dY, lddy, sw, P, pitch, planes, M, N);
  return 0;
}

int launch_finish(const float* acc, int64_t kp, int splits, const float* g, const int64_t* target,
                  int64_t nvocab, int type, void* dX, int64_t lddx, int M, int K,
                  hipStream_t st) {
  finish_kernel<<<(uint32_t)ceil_div((int64_t)M * K, 256), 256, 0, st>>>(
      acc, kp, splits, g, target, nvocab, type, dX, lddx, M, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
