// i8_block.h -- internal interface of what stands between the int8 products: the
// argument blocks and launchers behind i8_block_abi.hip.  Every launcher assumes
// validated arguments and returns 0, or -1 when the problem does not fit a grid.
// A `wide` flag says that every row of its matrix can be accessed 16 bytes at a time.
#pragma once

#include "i8.h"

namespace gemmq {
namespace i8 {

// i8_norm.hip
struct RmsArgs {
  const void *X, *R;  // R, H may be null
  void* H;
  const float* w;
  int8_t* Q;
  float* s;
  int64_t ldx, ldr, ldh, ldq;
  int type, M, K;
  float eps;
  bool wide_x, wide_r, wide_h, wide_w;
};
int launch_rms(const RmsArgs& a, hipStream_t st);

struct RmsGradArgs {
  const void *H, *dY, *dH;  // dH may be null
  const float* w;
  void* dX;
  float* part;  // [rms_grad_groups][kp], of one group dw itself; or null: no dw
  int64_t ldh, lddy, lddh, lddx, kp;  // kp: K rounded up to a multiple of 4, or K of dw itself
  int type, M, K;
  float eps;
  bool wide_h, wide_dy, wide_dh, wide_dx, wide_w, wide_part;
};
int rms_grad_groups(int64_t M, int64_t K);
int launch_rms_grad(const RmsGradArgs& a, hipStream_t st);

// out[k] = the sum of `count` rows of part, in a fixed order (count 0: zeros); and of a second
// one in the same launch, where it is not null
struct Join {
  const float* part;
  float* out;
};
int launch_join(Join a, Join b, int64_t pitch, int count, int K, hipStream_t st);

// The product with an activation, and the gated pair of products (i8_act.hip):
// y = act(z) (+ r), or act(z) u.  A matrix of results or residuals has 16-bit rows that
// can be accessed eight values at a time (`lines`, 16 bytes) and, in any type, four
// (`wide`).
struct Rows {
  void* p;  // null: left out
  int64_t ld;
  bool wide, lines;
};
struct ActOut {
  const float *bias, *biasu;  // may be null
  const int8_t* Wu;           // the second matrix of a pair, with its scales
  const float* swu;
  int64_t ldwu;
  Rows R, Y, Z, U;
  int act, type;
};
// rows of W that a launch goes through: N, 2 N of a pair (`pair`: of ActOut::Wu)
int launch_act(const Operands& op, const ActOut& out, bool pair, hipStream_t st);
bool act_fits(int M, int N, int K, bool pair);
bool act_fuses(int M, int N, int K, bool pair);
int launch_act_fused(int xtype, const void* X, int64_t ldx, const Operands& op, const ActOut& out,
                     bool pair, hipStream_t st);

// i8_act_grad.hip: dZ = dY act'(Z), or with U dZ = dY U act'(Z) and dU = dY act(Z);
// sums[0] and sums[1] (or null) receive the groups' sums over rows of dZ and dU, np apart.
struct ActGradArgs {
  Rows Z, U, dY, dZ, dU;  // U, dU null: no pair
  float* sums[2];
  int64_t np;
  int act, type, M, N, groups;
};
int act_grad_groups(int type, int64_t M, int64_t N);  // with sums over rows
int launch_act_grad(ActGradArgs a, hipStream_t st);

// i8_sample.hip: one token a row.  What the first launch leaves of a part of a row:
struct SamplePart {
  float top, low;  // its largest logit, its lowest finite one (-inf, +inf: none)
  uint32_t bad;    // a NaN or +inf
};
struct SampleArgs {
  const void* Z;
  int64_t ldz;
  const float *temperature, *top_p, *min_p;  // may be null
  const int32_t* top_k;                      // may be null
  const float* u;
  int64_t* token;
  float* logprob;  // may be null
  int N;
  bool wide;
  // set by the launcher: a part's logits and their number, the bits of a weight, and the
  // workspace
  int chunk, chunks, bits;
  SamplePart* part;
  double* sum;
  void* rows;
  uint32_t *count, *listed, *first;
  unsigned long long *weight, *list;
};
size_t sample_workspace(int64_t M, int64_t N);
int launch_sample(SampleArgs a, int type, int64_t M, void* ws, hipStream_t st);

}  // namespace i8
}  // namespace gemmq
