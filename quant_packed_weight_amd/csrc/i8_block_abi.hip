// i8_block_abi.hip -- the entry points of what stands between the int8 products
// (gemmq_i8.h): validation, workspace layout and the order of launches, as in
// i8_abi.hip.
#include "i8_block.h"
#include "i8_check.h"

using gemmq::aligned;
using gemmq::check_device;
using gemmq::clear_pending;
using gemmq::launched;
using namespace gemmq::i8;

namespace {

// an output that is an input itself lies in memory as the input does
bool same_rows(const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t M) {
  return out != in || !out || ldo == ldi || M == 1;
}

// a matrix that may be left out
int check_optional(int type, const void* p, int64_t ld, int64_t width) {
  return p ? check_rows(type, p, ld, width) : GEMMQ_OK;
}

bool eps_ok(float eps) { return eps >= 0.0f && eps < __builtin_inff(); }

}  // namespace

extern "C" {

int gemmq_rms_i8(int type, const void* X, int64_t ldx, const void* R, int64_t ldr, void* H,
                 int64_t ldh, const float* w, float eps, int8_t* Q, int64_t ldq, float* s,
                 int64_t M, int64_t K, void* stream) {
  int rc = check_shape(M, 0, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type) || !eps_ok(eps)) return GEMMQ_E_INVALID_ARG;
  if (M == 0) return GEMMQ_OK;
  rc = check_rows(type, X, ldx, K);
  if (rc == GEMMQ_OK) rc = check_optional(type, R, ldr, K);
  if (rc == GEMMQ_OK) rc = check_optional(type, H, ldh, K);
  if (rc == GEMMQ_OK) rc = check_i8(Q, ldq, s, K);
  if (rc == GEMMQ_OK && !w) rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK && !aligned(w, 4)) rc = GEMMQ_E_ALIGNMENT;
  if (rc == GEMMQ_OK && !(same_rows(H, ldh, X, ldx, M) && same_rows(H, ldh, R, ldr, M)))
    rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  const RmsArgs a{X,   R,   H,   w,    Q,      s,      ldx,  ldr,
                  ldh, ldq, type, (int)M, (int)K, eps,
                  wide_rows(X, ldx, type), wide_rows(R, ldr, type), wide_rows(H, ldh, type),
                  aligned(w, 16)};
  clear_pending();
  return launched(launch_rms(a, static_cast<hipStream_t>(stream)));
}

size_t gemmq_rms_i8_grad_workspace(int type, int64_t M, int64_t K) {
  if (!known(type) || check_shape(M, 0, K) != GEMMQ_OK || M == 0) return 0;
  return align_up(4 * rms_grad_groups(M) * (int64_t)align_up(K, 4), 256);
}

int gemmq_rms_i8_grad(int type, const void* H, int64_t ldh, const float* w, float eps,
                      const void* dY, int64_t lddy, const void* dH, int64_t lddh, void* dX,
                      int64_t lddx, float* dw, int64_t M, int64_t K, void* ws, size_t ws_bytes,
                      void* stream) {
  int rc = check_shape(M, 0, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type) || !eps_ok(eps)) return GEMMQ_E_INVALID_ARG;
  if (!aligned(dw, 4)) return GEMMQ_E_ALIGNMENT;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M == 0) {
    if (!dw) return GEMMQ_OK;
    rc = check_device();
    if (rc != GEMMQ_OK) return rc;
    clear_pending();
    return launched(launch_join(nullptr, 0, 0, dw, (int)K, st));
  }
  rc = check_rows(type, H, ldh, K);
  if (rc == GEMMQ_OK) rc = check_rows(type, dY, lddy, K);
  if (rc == GEMMQ_OK) rc = check_optional(type, dH, lddh, K);
  if (rc == GEMMQ_OK) rc = check_rows(type, dX, lddx, K);
  if (rc == GEMMQ_OK && !w) rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK && !aligned(w, 4)) rc = GEMMQ_E_ALIGNMENT;
  if (rc == GEMMQ_OK && !(same_rows(dX, lddx, dY, lddy, M) && same_rows(dX, lddx, dH, lddh, M)))
    rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK && dw) rc = check_ws(ws, ws_bytes, gemmq_rms_i8_grad_workspace(type, M, K));
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  const int64_t kp = (int64_t)align_up(K, 4);
  float* part = dw ? static_cast<float*>(ws) : nullptr;
  const RmsGradArgs a{H,    dY,   dH,   w,    dX,     part,   ldh,
                      lddy, lddh, lddx, kp,   type,   (int)M, (int)K,
                      eps,  wide_rows(H, ldh, type),  wide_rows(dY, lddy, type),
                      wide_rows(dH, lddh, type),      wide_rows(dX, lddx, type),
                      aligned(w, 16)};
  clear_pending();
  rc = launched(launch_rms_grad(a, st));
  if (rc != GEMMQ_OK || !dw) return rc;
  return launched(launch_join(part, kp, rms_grad_groups(M), dw, (int)K, st));
}

}  // extern "C"
