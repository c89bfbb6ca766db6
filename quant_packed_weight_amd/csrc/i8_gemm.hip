// i8_gemm.hip -- launches of the int8 product by tiles (i8_tile.h) for the linear layer,
// the vocabulary loss and its gradient's softmax factor, and the join of the loss.
#include "i8_tile.h"

namespace gemmq {
namespace i8 {
namespace {

// The tiles of each row joined by log-sum-exp, and the target's logit from its
// own row of the weights (the same exact sum as in the tile that held it): one
// workgroup per row.
__global__ __launch_bounds__(256) void loss_join_kernel(Operands op, LossOut o, float* loss,
                                                        float* lse) {
  __shared__ float tops[4], sums[4];
  __shared__ int dots[4];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t m = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  if (m >= op.M) return;  // all of the workgroup
  const float2* p = o.part + m * o.ntiles;
  const int64_t tg = o.target[m];
  const bool hit = tg >= 0 && tg < op.N;
  int dot = 0;
  if (hit) {
    const int8_t *x = op.X + m * op.ldx, *w = op.W + tg * op.ldw;
    for (int k = 16 * t; k < op.K; k += 4096) {
      const v4i a = keep_bytes(*reinterpret_cast<const v4i*>(x + k), op.K - k);
      const v4i b = *reinterpret_cast<const v4i*>(w + k);
#pragma unroll
      for (int c = 0; c < 4; ++c) dot = __builtin_amdgcn_sdot4(a[c], b[c], dot, false);
    }
  }
  float top = -__builtin_inff();
  for (int i = t; i < o.ntiles; i += 256) top = fmaxf(top, p[i].x);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    top = fmaxf(top, __shfl_xor(top, d, 64));
    dot += __shfl_xor(dot, d, 64);
  }
  if (lane == 0) {
    tops[wave] = top;
    dots[wave] = dot;
  }
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  float sum = 0.0f;
  const float sx = op.sx[m], size = fabsf(sx), s2 = size * kLog2e;
  for (int i = t; i < o.ntiles; i += 256) sum += join_term(p[i], top, s2);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (t == 0) {
    // lse = z(top) + log(sum): the large one of the two is a product, carried with its
    // remainder and rounded once with the rest.  (From base 2, top log2 e and back, lse
    // was two to three times as far off as its rounding, and 1 - p of a certain row with
    // it.)  The target's logit is taken from the maximum before anything of the two's
    // size is rounded.  What the target's v leaves of its logit (and the other columns' of
    // theirs: not known here) counts in lse by its probability and in the loss by the rest.
    const float rest = __builtin_log2f((sums[0] + sums[1]) + (sums[2] + sums[3])) * kLn2;
    const float high = top * size, low = fmaf(top, size, -high);
    float below = __builtin_nanf(""), off = 0.0f;
    if (hit) {
      float left;
      const float v = scaled((dots[0] + dots[1]) + (dots[2] + dots[3]), op.sw[tg], left);
      below = fmaf(sx < 0.0f ? top + v : top - v, size, rest);
      const float p = __expf(-below);
      off = left * sx * p;
      below -= left * sx * (1.0f - p);
    }
    lse[m] = high + (low + rest + off);
    loss[m] = tg < 0 ? 0.0f : below;
  }
}

}  // namespace

bool product_fits(int M, int N, int K) {
  return grid_fits(tiles(kTiles[pick_tile(M, N, K)], M, N), kMaxThreads);
}

int launch_linear(const Operands& op, const LinearOut& out, hipStream_t st) {
  if (skinny(op.M, op.N, true)) return launch_skinny(op, out, st);
  TileArgs a{};
  a.op = op;
  a.lin = out;
  return launch_tiles<kLinear>(a, st);
}

int loss_tiles(int M, int N, int K) {
  const int width = skinny(M, N, false) ? kSkinnyChannels : kTiles[pick_tile(M, N, K)].bn;
  return (int)ceil_div(N, width);
}

int launch_loss(const Operands& op, const LossOut& out, hipStream_t st) {
  if (skinny(op.M, op.N, false)) return launch_skinny(op, out, st);
  TileArgs a{};
  a.op = op;
  a.loss = out;
  return launch_tiles<kLoss>(a, st);
}

int launch_loss_join(const Operands& op, const LossOut& o, float* loss, float* lse,
                     hipStream_t st) {
  loss_join_kernel<<<rows_grid(1, op.M), 256, 0, st>>>(op, o, loss, lse);
  return 0;
}

int launch_factor(const Operands& op, const FactorOut& out, hipStream_t st) {
  if (skinny(op.M, op.N, false)) return launch_skinny(op, out, st);
  TileArgs a{};
  a.op = op;
  a.fac = out;
  return launch_tiles<kFactor>(a, st);
}

}  // namespace i8
}  // namespace gemmq
