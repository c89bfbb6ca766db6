// i8.h -- internal interface of the int8 half (gemmq_i8.h): the argument blocks
// and launchers behind i8_abi.hip.  Every launcher assumes validated arguments
// and returns 0, or -1 when the problem does not fit a grid.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemmq_i8.h"

namespace gemmq {
namespace i8 {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t type_bytes(int type) { return type == GEMMQ_F32 ? 4 : 2; }

// a launch holds fewer than 2^32 threads in a dimension
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks * threads < (1LL << 32); }
// x workgroups for each of M rows, the rows over the second and third dimensions
// (a kernel's row is blockIdx.y + gridDim.y * blockIdx.z, and may lie past M)
inline dim3 rows_grid(int64_t x, int64_t M) {
  const int64_t y = M < 32768 ? M : 32768;
  return dim3((uint32_t)x, (uint32_t)y, (uint32_t)ceil_div(M, y));
}

// whether every row of a matrix can be read 16 bytes at a time from its first value
inline bool wide_rows(const void* p, int64_t ld, int type) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * type_bytes(type) % 16 == 0;
}

// bf16 numbers that carry one value of `type` in the gradient's products
// (8 significant bits each): all of a bf16, f16's 11 bits, all of an f32.  The one of bf16
// is a rounding of dy sw (or sw w, or the softmax factor) beside the result's own: its
// errors average out over N and the result is off by 2.35e-3 instead of 1.66e-3 in the
// norm, where a second number costs half again the product's time (M = 2048, 4096 x 4096
// 74 us, two 112, three 152).  See grad_planes for few rows.
inline int planes_of(int type) { return type == GEMMQ_BF16 ? 1 : type == GEMMQ_F16 ? 2 : 3; }

// The int8 operands: sum over k of X[m, k] * W[n, k] for m < M, n < N, and
// their scales.
struct Operands {
  const int8_t* W;
  const float* sw;
  const int8_t* X;
  const float* sx;
  int64_t ldw, ldx;
  int M, N, K;
};

// y = sx sw I (+ bias)
struct LinearOut {
  const float* bias;
  void* Y;
  int64_t ldy;
  int type;
  bool wide;   // four consecutive values of a row may be stored at once
  bool lines;  // of 16 bits, and eight may
};

// Softmax statistics per column tile: of row m in tile t, with v = sw I and the sign of
// sx, (max v, sum of exp(|sx| (v - max v))) at part[m * ntiles + t].
struct LossOut {
  const int64_t* target;
  float2* part;
  int ntiles;
};

// The softmax factor (exp(z - lse) - [n == target]) * sw of one piece of the
// vocabulary (operands' row 0 is vocabulary row n0) as `planes` bf16 matrices of
// [M, pitch], plane p at P + p * M * pitch; columns from N to the pitch are zero.
struct FactorOut {
  const int64_t* target;
  const float* lse;
  uint16_t* P;
  int64_t pitch, n0;
  int planes;
  float* rest;  // [M], or null: what one plane's rounding leaves of the target's value
};

int launch_quantize(int type, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s, int M,
                    int K, hipStream_t st);

// i8_gemm.hip: the product by tiles in LDS, or by i8_skinny.hip's stream of W where
// that is faster; each with its own check of the grid
bool product_fits(int M, int N, int K);
int launch_linear(const Operands& op, const LinearOut& out, hipStream_t st);
int loss_tiles(int M, int N, int K);  // column tiles of the loss launch (LossOut::ntiles)
int launch_loss(const Operands& op, const LossOut& out, hipStream_t st);
int launch_loss_join(const Operands& op, const LossOut& o, float* loss, float* lse,
                     hipStream_t st);
int launch_factor(const Operands& op, const FactorOut& out, hipStream_t st);

// i8_skinny.hip, M <= kSkinnyMaxM
constexpr int kSkinnyMaxM = 16, kSkinnyChannels = 16;  // channels per workgroup
int launch_skinny(const Operands& op, const LinearOut& out, hipStream_t st);
int launch_skinny(const Operands& op, const LossOut& out, hipStream_t st);
int launch_skinny(const Operands& op, const FactorOut& out, hipStream_t st);
// the layer in one launch: X quantized by every workgroup, one writes op.X and op.sx
bool fuses(int M, int N, int K);
int launch_fused(int xtype, const void* X, int64_t ldx, const Operands& op, const LinearOut& out,
                 hipStream_t st);

// i8_grad.hip: v[m, k] = sum over n of (sum of planes)[m, n] * W[n, k], by ranges
// of n: range s gives acc[s][m][k] (+)= its sum, which launch_finish adds up, or,
// where there is one range and one piece (acc null), the result itself.
struct GradOut {
  // dX[m] = v[m] * g[m] (g null: 1), zero where target[m] < 0 and NaN where it is
  // nvocab or more (target null: neither)
  const float* g;
  const int64_t* target;
  int64_t nvocab;
  int type;
  void* dX;
  int64_t lddx;
  bool wide;  // four consecutive values of a row may be stored at once
  const float* rest;  // not null: rest[m] * (row target[m] of W) is added to v[m]
  const int8_t* W;    // (with rest) all rows, as the entry point has them
  int64_t ldw;
};
struct GradArgs {
  const int8_t* W;     // the piece's first row
  int64_t ldw;
  const uint16_t* P;   // planes of [M, pitch]; or, with sw, one matrix of the caller's
  int64_t pitch;       // a multiple of 64 (of 8, N too, with sw)
  float* acc;          // [splits][M][kp], or null
  int64_t kp;          // pitch of a row of acc, a multiple of 4, >= K
  int M, N, K, planes;
  int tile, splits;    // of grad_split
  bool add;            // add to what acc holds (a later piece)
  const float* sw;     // not null (M <= 128): scales W's rows, or with two planes (M <= 8)
                       // the caller's matrix, as two bf16 numbers
  GradOut out;
};
struct GradSplit {
  int tile, splits;
};
// the tile and the ranges for pieces of N columns; `whole`: there is one piece
GradSplit grad_split(int M, int N, int K, int planes, bool whole);
bool grad_fits(const GradSplit& s, int M, int K);
int launch_grad(const GradArgs& a, hipStream_t st);

// planes of dY * sw for columns [n0, n0 + N) of dY; columns up to the pitch zero
int launch_planes(int type, const void* dY, int64_t lddy, const float* sw, uint16_t* P,
                  int64_t pitch, int planes, int M, int N, hipStream_t st);

int launch_finish(const float* acc, int64_t kp, int splits, const GradOut& out, int M, int K,
                  hipStream_t st);

}  // namespace i8
}  // namespace gemmq
