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
  float* part;  // [rms_grad_groups][kp], or null: no dw
  int64_t ldh, lddy, lddh, lddx, kp;  // kp: K rounded up to a multiple of 4
  int type, M, K;
  float eps;
  bool wide_h, wide_dy, wide_dh, wide_dx, wide_w;
};
int rms_grad_groups(int64_t M);
int launch_rms_grad(const RmsGradArgs& a, hipStream_t st);

// out[k] = the sum of `count` rows of part, in a fixed order (count 0: zeros)
int launch_join(const float* part, int64_t pitch, int count, float* out, int K, hipStream_t st);

}  // namespace i8
}  // namespace gemmq
