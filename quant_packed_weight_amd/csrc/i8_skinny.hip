// i8_skinny.hip -- the int8 product for few tokens (M <= 16): a stream of W
// straight into registers, with the same three epilogues as i8_gemm.hip and, for
// the linear layer at decode sizes, the quantizer in the same launch.
//
// I[n, m] on 16 x 16 x 64 MFMAs: 16 rows of W by 64 bytes of K are one 16-byte
// load per lane, as the instruction wants them, so W passes through no LDS; 16
// tokens stand at the other operand, also for M = 1, where the products are idle
// but no sum across lanes is needed.  A workgroup takes 16 channels, its waves
// alternate 128-byte pieces of K and add their sums through LDS.  Bound by the
// read of W; the activations' reads from L2, as many bytes as W's for each 16
// tokens, are why more tokens go to tiles in LDS (i8_gemm.hip).  16, 32 or 64
// channels a workgroup (fewer such reads, fewer workgroups): N = K = 4096 at M = 8
// 5.9 / 8.1 / 12.4 us, 151936 x 2048 at M = 1 53 / 54 / 59.
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

constexpr int kPiece = 128;  // bytes of K per load pair: whole lines of W
// the fused form: tokens, and bytes of int8 activations that a workgroup holds
constexpr int kFusedRows = 2, kFusedBytes = 16384;

struct SkinnyArgs {
  Operands op;
  LinearOut lin;
  LossOut loss;
  FactorOut fac;
  const void* X;  // fused: the activations, quantized here and written to op.X, op.sx
  int64_t ldx;
  int xtype;
  bool xwide;  // 16-byte loads from its rows
};

__device__ __forceinline__ v4i mfma16(v4i a, v4i b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// The activations quantized by the whole workgroup into xl (LDS, `span` bytes a
// row, zero from column K on) and their scales into xs: the steps of
// i8_quantize.hip.
template <int TYPE, int T>
__device__ __forceinline__ void quantize_rows(const SkinnyArgs& a, int span, uint8_t* xl, float* xs,
                                              uint32_t (*tops)[16], int t) {
  constexpr int V = TYPE == GEMMQ_F32 ? 4 : 8;
  const Operands& op = a.op;
  for (int m = 0; m < op.M; ++m) {
    uint32_t top = 0;
    for (int k = V * t; k < op.K; k += V * T) {
      float v[V];
      load_values<TYPE, V>(a.X, m * a.ldx + k, op.K - k, a.xwide, v);
#pragma unroll
      for (int e = 0; e < V; ++e) top = max(top, abs_bits(v[e]));
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
    if ((t & 63) == 0) tops[m][t >> 6] = top;
  }
  __syncthreads();
  for (int m = 0; m < op.M; ++m) {
    uint32_t top = tops[m][0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) top = max(top, tops[m][w]);
    const float s = scale_of(top);
    const float inv = 1.0f / s;
    if (t == 0) xs[m] = s;
    for (int k = V * t; k < span; k += V * T) {
      float v[V];
      load_values<TYPE, V>(a.X, m * a.ldx + k, op.K - k, a.xwide, v);
      uint32_t q[V / 4];
      quantize_values<V>(v, s, inv, q);
#pragma unroll
      for (int w = 0; w < V / 4; ++w)
        *reinterpret_cast<uint32_t*>(xl + m * span + k + 4 * w) = q[w];
    }
  }
  __syncthreads();
}

template <int KS, int DEPTH, int EPI, bool FUSED>
__global__ __launch_bounds__(64 * KS) void skinny_kernel(SkinnyArgs a) {
  constexpr int T = 64 * KS;
  __shared__ __attribute__((aligned(16))) v4i sums[KS * 64];
  __shared__ __attribute__((aligned(16))) uint8_t xl[FUSED ? kFusedBytes : 16];
  __shared__ float xs[16];
  __shared__ uint32_t tops[FUSED ? kFusedRows : 1][16];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const Operands& op = a.op;
  const int64_t n0 = (int64_t)xcd_order(blockIdx.x, gridDim.x) * 16;
  const int row = lane & 15, part = 16 * (lane >> 4);
  const int last = (op.K - 1) / 16 * 16;  // the 16 bytes that hold column K - 1
  const int pieces = (op.K + kPiece - 1) / kPiece;

  // rows past the last channel or token repeat it, bytes past column K the last 16
  const int8_t* wp = op.W + min(n0 + row, (int64_t)op.N - 1) * op.ldw;
  const int8_t* xp = op.X + min(row, op.M - 1) * op.ldx;

  v4i wf[DEPTH][2], xf[FUSED ? 1 : DEPTH][2];
  auto load = [&](int u, int i) {
    const int k0 = min(wave + KS * i, pieces - 1) * kPiece;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int k = min(k0 + 64 * half + part, last);
      wf[u][half] = *reinterpret_cast<const v4i*>(wp + k);
      if constexpr (!FUSED) xf[u][half] = *reinterpret_cast<const v4i*>(xp + k);
    }
  };
  v4i acc = {0, 0, 0, 0};
  const int span = pieces * kPiece;
  auto multiply = [&](int u, int i) {
    const int piece = wave + KS * i;
    if constexpr (FUSED) {
      if (piece >= pieces) return;
#pragma unroll
      for (int half = 0; half < 2; ++half)
        xf[0][half] = *reinterpret_cast<const v4i*>(xl + min(row, op.M - 1) * span +
                                                    piece * kPiece + 64 * half + part);
    } else if (piece * kPiece + kPiece > op.K) {
      // the activations are zero from column K on, and in a piece past the last one
#pragma unroll
      for (int half = 0; half < 2; ++half)
        xf[u][half] = keep_bytes(xf[u][half], op.K - (piece * kPiece + 64 * half + part));
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) acc = mfma16(wf[u][half], xf[FUSED ? 0 : u][half], acc);
  };

  const int rounds = (pieces + KS - 1) / KS;
#pragma unroll
  for (int u = 0; u < DEPTH; ++u) load(u, u);
  if constexpr (FUSED) {
    if (a.xtype == GEMMQ_F32)
      quantize_rows<GEMMQ_F32, T>(a, span, xl, xs, tops, t);
    else if (a.xtype == GEMMQ_BF16)
      quantize_rows<GEMMQ_BF16, T>(a, span, xl, xs, tops, t);
    else
      quantize_rows<GEMMQ_F16, T>(a, span, xl, xs, tops, t);
    if (blockIdx.x == 0) {
      // the caller's copy, 16 bytes at a time but for a row's last ones
      const int chunks = (op.K + 15) / 16;
      for (int i = t; i < op.M * chunks; i += T) {
        const int m = i / chunks, k = i % chunks * 16;
        int8_t* q = const_cast<int8_t*>(op.X) + m * op.ldx + k;
        const uint8_t* from = xl + m * span + k;
        if (k + 16 <= op.K)
          *reinterpret_cast<v4i*>(q) = *reinterpret_cast<const v4i*>(from);
        else
          for (int e = 0; k + e < op.K; ++e) q[e] = (int8_t)from[e];
      }
      if (t < op.M) const_cast<float*>(op.sx)[t] = xs[t];
    }
  } else {
    if (t < 16) xs[t] = t < op.M ? op.sx[t] : 0.0f;
  }
  // a group of DEPTH rounds at a time: the loads of the next group are issued as
  // this one's registers come free; rounds past the last piece add zero
  for (int i = 0; i < rounds; i += DEPTH) {
    if (i + DEPTH < rounds) {
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) {
        multiply(u, i + u);
        load(u, i + DEPTH + u);
      }
    } else {
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) multiply(u, i + u);
    }
  }

  sums[wave * 64 + lane] = acc;
  __syncthreads();

  // lane l holds token l & 15 and channels 4 (l >> 4) + 0..3
  if (wave > 0) return;
  v4i s = sums[lane];
#pragma unroll
  for (int w = 1; w < KS; ++w) s += sums[w * 64 + lane];
  const int m = row;
  const int64_t n = n0 + 4 * (lane >> 4);
  const bool inside = m < op.M;
  const int count = (int)min((int64_t)4, op.N - n);  // channels of these four that exist
  const float sx = xs[m];
  float sw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sw[e] = e < count ? op.sw[n + e] : 0.0f;
  if constexpr (EPI == kLinear) {
    if (!inside) return;
    float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.lin.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = e < count ? a.lin.bias[n + e] : 0.0f;
    }
    store4_as(a.lin.Y, m * a.lin.ldy + n, a.lin.type, a.lin.wide, count,
              fmaf((float)s[0] * sx, sw[0], b[0]), fmaf((float)s[1] * sx, sw[1], b[1]),
              fmaf((float)s[2] * sx, sw[2], b[2]), fmaf((float)s[3] * sx, sw[3], b[3]));
  } else if constexpr (EPI == kFactor) {
    if (!inside || n >= a.fac.pitch) return;  // the pitch is a multiple of 4
    const float lse = a.fac.lse[m];
    const int64_t tg = a.fac.target[m] - a.fac.n0 - n;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float p = __builtin_amdgcn_exp2f(fmaf((float)s[e] * sw[e], sx, -lse) * kLog2e);
      if (tg == e) p = target_factor(s[e], sw[e], sx, lse);
      f[e] = e < count ? p * sw[e] : 0.0f;
      if (tg == e && e < count && a.fac.rest) a.fac.rest[m] = bf16_rest(f[e]);
    }
    store_planes(a.fac.P + m * a.fac.pitch + n, (int64_t)op.M * a.fac.pitch, a.fac.planes, f);
  } else {
    // (max, sum) of a token over the 16 channels, as in i8_gemm.hip; the first of
    // them exists, so there is a maximum
    const float s2 = fabsf(sx) * kLog2e;
    float v[4], top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = (float)s[e] * (sx < 0.0f ? -sw[e] : sw[e]);
      if (e < count) top = fmaxf(top, v[e]);
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < count) sum += __builtin_amdgcn_exp2f((v[e] - top) * s2);
    sum += __shfl_xor(sum, 16, 64);
    sum += __shfl_xor(sum, 32, 64);
    if (inside && lane < 16)
      a.loss.part[(int64_t)m * a.loss.ntiles + n0 / kSkinnyChannels] = make_float2(top, sum);
  }
}

template <int EPI>
int launch(SkinnyArgs& a, hipStream_t st) {
  // the factor's columns up to its pitch are written, zero from N on
  const int64_t n = ceil_div(EPI == kFactor ? a.fac.pitch : a.op.N, kSkinnyChannels);
  if (!grid_fits(n, 1024)) return -1;
  const dim3 grid((uint32_t)n);
  // The more workgroups, the fewer waves need to share a channel's K (us, eight
  // waves / four: M = 8, 4096 x 4096 5.9 / 6.2, 12288 x 4096 14.4 / 13.5; M = 16,
  // 16384 x 2048 12.9 / 11.5), and beyond 2048, which only the linear layer has,
  // the more loads each may hold (151936 x 2048 at M = 4: 57, eight waves 61).
  if constexpr (EPI == kLinear) {
    if (n > 2048) {
      skinny_kernel<4, 4, EPI, false><<<grid, 256, 0, st>>>(a);
      return 0;
    }
  }
  if (n > 512)
    skinny_kernel<4, 2, EPI, false><<<grid, 256, 0, st>>>(a);
  else
    skinny_kernel<8, 2, EPI, false><<<grid, 512, 0, st>>>(a);
  return 0;
}

}  // namespace

int launch_skinny(const Operands& op, const LinearOut& out, hipStream_t st) {
  SkinnyArgs a{};
  a.op = op;
  a.lin = out;
  return launch<kLinear>(a, st);
}

int launch_skinny(const Operands& op, const LossOut& out, hipStream_t st) {
  SkinnyArgs a{};
  a.op = op;
  a.loss = out;
  return launch<kLoss>(a, st);
}

int launch_skinny(const Operands& op, const FactorOut& out, hipStream_t st) {
  SkinnyArgs a{};
  a.op = op;
  a.fac = out;
  return launch<kFactor>(a, st);
}

bool fuses(int M, int N, int K) {
  return M <= kFusedRows && (M == 1 || N <= 16384) &&
         M * ceil_div(K, kPiece) * kPiece <= kFusedBytes;
}

int launch_fused(int xtype, const void* X, int64_t ldx, const Operands& op, const LinearOut& out,
                 hipStream_t st) {
  SkinnyArgs a{};
  a.op = op;
  a.lin = out;
  a.X = X;
  a.ldx = ldx;
  a.xtype = xtype;
  a.xwide = wide_rows(X, ldx, xtype);
  const int64_t n = ceil_div(op.N, kSkinnyChannels);
  if (!grid_fits(n, 1024)) return -1;
  const dim3 grid((uint32_t)n);
  // The more waves, the sooner the workgroup has its activations; the more
  // workgroups, the less that matters: M = 1, 16, 8 and 4 waves, N = K = 4096 6.6 /
  // 6.9 / 7.6 us, 12288 x 4096 16.2 / 13.4 / 14.6, 151936 x 2048 132 / 89 / 54.
  if (n <= 512)
    skinny_kernel<16, 2, kLinear, true><<<grid, 1024, 0, st>>>(a);
  else if (n <= 2048)
    skinny_kernel<8, 4, kLinear, true><<<grid, 512, 0, st>>>(a);
  else
    skinny_kernel<4, 4, kLinear, true><<<grid, 256, 0, st>>>(a);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
