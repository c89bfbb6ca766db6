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

bool known_act(int act) { return act >= GEMMQ_ACT_NONE && act <= GEMMQ_ACT_RELU; }

Rows rows(int type, const void* p, int64_t ld) {
  return {const_cast<void*>(p), ld, ld % 4 == 0 && aligned(p, (uintptr_t)(4 * type_bytes(type))),
          wide_rows(p, ld, type)};
}

// A second int8 matrix, its scales and its bias, and what receives its products
struct Pair {
  const int8_t* W;
  int64_t ldw;
  const float *sw, *bias;
  void* U;
  int64_t ldu;
};

// Everything of a product with an activation (pair null) or of a gated pair but the
// quantizer's input; `empty` where there is nothing to compute.
int check_act(const int8_t* W, int64_t ldw, const float* sw, const Pair* pair, const int8_t* Xq,
              int64_t ldq, const float* sx, const float* bias, int act, const void* R, int64_t ldr,
              int ytype, void* Y, int64_t ldy, void* Z, int64_t ldz, int64_t M, int64_t N,
              int64_t K, Operands& op, ActOut& out, bool& empty) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(ytype) || !known_act(act)) return GEMMQ_E_INVALID_ARG;
  empty = M == 0 || N == 0;
  if (empty) return GEMMQ_OK;
  rc = check_i8(W, ldw, sw, K);
  if (rc == GEMMQ_OK && pair) rc = check_i8(pair->W, pair->ldw, pair->sw, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc == GEMMQ_OK) rc = check_rows(ytype, Y, ldy, N);
  if (rc == GEMMQ_OK) rc = check_optional(ytype, R, ldr, N);
  if (rc == GEMMQ_OK) rc = check_optional(ytype, Z, ldz, N);
  if (rc == GEMMQ_OK && pair) rc = check_optional(ytype, pair->U, pair->ldu, N);
  if (rc != GEMMQ_OK) return rc;
  if (!aligned(bias, 4) || (pair && !aligned(pair->bias, 4))) return GEMMQ_E_ALIGNMENT;
  const void* U = pair ? pair->U : nullptr;
  if (!same_rows(Y, ldy, R, ldr, M) || Y == Z || Y == U || (Z && (Z == U || Z == R)))
    return GEMMQ_E_INVALID_ARG;
  if (!act_fits((int)M, (int)N, (int)K, pair != nullptr)) return GEMMQ_E_SHAPE;
  op = Operands{W, sw, Xq, sx, ldw, ldq, (int)M, (int)N, (int)K};
  out = ActOut{};
  out.bias = bias;
  out.R = rows(ytype, R, ldr);
  out.Y = rows(ytype, Y, ldy);
  out.Z = rows(ytype, Z, ldz);
  out.act = act;
  out.type = ytype;
  if (pair) {
    out.biasu = pair->bias;
    out.Wu = pair->W;
    out.ldwu = pair->ldw;
    out.swu = pair->sw;
    out.U = rows(ytype, pair->U, pair->ldu);
  }
  return GEMMQ_OK;
}

int run_gemm(const Operands& op, const ActOut& out, bool pair, hipStream_t st) {
  const int rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  clear_pending();
  return launched(launch_act(op, out, pair, st));
}

// whether a result lies in X's place
bool in_place(int xtype, const void* X, int64_t ldx, const Operands& op, const ActOut& out) {
  const Span x = span(xtype, X, ldx, op.K);
  for (const Rows* r : {&out.Y, &out.Z, &out.U})
    if (share_memory(x, span(out.type, r->p, r->ld, op.N), op.M)) return true;
  return false;
}

// the same with the quantizer before it or in the same launch
int run_linear(int xtype, const void* X, int64_t ldx, int8_t* Xq, int64_t ldq, float* sx, int64_t M,
               int64_t K, bool empty, const Operands& op, const ActOut& out, bool pair,
               hipStream_t st) {
  if (!known(xtype)) return GEMMQ_E_INVALID_ARG;
  if (M == 0) return GEMMQ_OK;
  int rc = check_rows(xtype, X, ldx, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  clear_pending();
  if (!empty && act_fuses(op.M, op.N, op.K, pair) && !in_place(xtype, X, ldx, op, out))
    return launched(launch_act_fused(xtype, X, ldx, op, out, pair, st));
  rc = launched(launch_quantize(xtype, X, ldx, Xq, ldq, sx, (int)M, (int)K, st));
  if (rc != GEMMQ_OK || empty) return rc;
  return launched(launch_act(op, out, pair, st));
}

// a workspace where one is needed
int check_need(const void* ws, size_t have, size_t need) {
  return need > 0 ? check_ws(ws, have, need) : GEMMQ_OK;
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
  const int64_t groups = rms_grad_groups(M, K);
  return groups > 1 ? align_up(4 * groups * (int64_t)align_up(K, 4), 256) : 0;
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
    return launched(launch_join({nullptr, dw}, {}, 0, 0, (int)K, st));
  }
  rc = check_rows(type, H, ldh, K);
  if (rc == GEMMQ_OK) rc = check_rows(type, dY, lddy, K);
  if (rc == GEMMQ_OK) rc = check_optional(type, dH, lddh, K);
  if (rc == GEMMQ_OK) rc = check_rows(type, dX, lddx, K);
  if (rc == GEMMQ_OK && !w) rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK && !aligned(w, 4)) rc = GEMMQ_E_ALIGNMENT;
  if (rc == GEMMQ_OK && !(same_rows(dX, lddx, dY, lddy, M) && same_rows(dX, lddx, dH, lddh, M) &&
                          same_rows(dX, lddx, H, ldh, M)))
    rc = GEMMQ_E_INVALID_ARG;
  if (rc == GEMMQ_OK && dw) rc = check_need(ws, ws_bytes, gemmq_rms_i8_grad_workspace(type, M, K));
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  const int groups = rms_grad_groups(M, K);
  const bool join = dw && groups > 1;  // else the kernel's sums are dw
  const int64_t kp = join ? (int64_t)align_up(K, 4) : K;
  float* part = join ? static_cast<float*>(ws) : dw;
  const RmsGradArgs a{H,    dY,   dH,   w,    dX,     part,   ldh,
                      lddy, lddh, lddx, kp,   type,   (int)M, (int)K,
                      eps,  wide_rows(H, ldh, type),  wide_rows(dY, lddy, type),
                      wide_rows(dH, lddh, type),      wide_rows(dX, lddx, type),
                      aligned(w, 16),                 kp % 4 == 0 && aligned(part, 16)};
  clear_pending();
  rc = launched(launch_rms_grad(a, st));
  if (rc != GEMMQ_OK || !join) return rc;
  return launched(launch_join({part, dw}, {}, kp, groups, (int)K, st));
}

int gemmq_gemm_i8_act(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Xq, int64_t ldq,
                      const float* sx, const float* bias, int act, const void* R, int64_t ldr,
                      int ytype, void* Y, int64_t ldy, void* Z, int64_t ldz, int64_t M, int64_t N,
                      int64_t K, void* stream) {
  Operands op;
  ActOut out;
  bool empty;
  const int rc = check_act(W, ldw, sw, nullptr, Xq, ldq, sx, bias, act, R, ldr, ytype, Y, ldy, Z,
                           ldz, M, N, K, op, out, empty);
  if (rc != GEMMQ_OK || empty) return rc;
  return run_gemm(op, out, false, static_cast<hipStream_t>(stream));
}

int gemmq_linear_i8_act(const int8_t* W, int64_t ldw, const float* sw, int xtype, const void* X,
                        int64_t ldx, int8_t* Xq, int64_t ldq, float* sx, const float* bias,
                        int act, const void* R, int64_t ldr, int ytype, void* Y, int64_t ldy,
                        void* Z, int64_t ldz, int64_t M, int64_t N, int64_t K, void* stream) {
  Operands op;
  ActOut out;
  bool empty;
  const int rc = check_act(W, ldw, sw, nullptr, Xq, ldq, sx, bias, act, R, ldr, ytype, Y, ldy, Z,
                           ldz, M, N, K, op, out, empty);
  if (rc != GEMMQ_OK) return rc;
  return run_linear(xtype, X, ldx, Xq, ldq, sx, M, K, empty, op, out, false,
                    static_cast<hipStream_t>(stream));
}

int gemmq_gemm_i8_gate(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Wu,
                       int64_t ldwu, const float* swu, const int8_t* Xq, int64_t ldq,
                       const float* sx, const float* bias, const float* biasu, int act, int ytype,
                       void* Y, int64_t ldy, void* Z, int64_t ldz, void* U, int64_t ldu, int64_t M,
                       int64_t N, int64_t K, void* stream) {
  Operands op;
  ActOut out;
  bool empty;
  const Pair pair{Wu, ldwu, swu, biasu, U, ldu};
  const int rc = check_act(W, ldw, sw, &pair, Xq, ldq, sx, bias, act, nullptr, 0, ytype, Y, ldy, Z,
                           ldz, M, N, K, op, out, empty);
  if (rc != GEMMQ_OK || empty) return rc;
  return run_gemm(op, out, true, static_cast<hipStream_t>(stream));
}

int gemmq_linear_i8_gate(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Wu,
                         int64_t ldwu, const float* swu, int xtype, const void* X, int64_t ldx,
                         int8_t* Xq, int64_t ldq, float* sx, const float* bias, const float* biasu,
                         int act, int ytype, void* Y, int64_t ldy, void* Z, int64_t ldz, void* U,
                         int64_t ldu, int64_t M, int64_t N, int64_t K, void* stream) {
  Operands op;
  ActOut out;
  bool empty;
  const Pair pair{Wu, ldwu, swu, biasu, U, ldu};
  const int rc = check_act(W, ldw, sw, &pair, Xq, ldq, sx, bias, act, nullptr, 0, ytype, Y, ldy, Z,
                           ldz, M, N, K, op, out, empty);
  if (rc != GEMMQ_OK) return rc;
  return run_linear(xtype, X, ldx, Xq, ldq, sx, M, K, empty, op, out, true,
                    static_cast<hipStream_t>(stream));
}

size_t gemmq_act_grad_workspace(int type, int64_t M, int64_t N) {
  if (!known(type) || check_shape(M, N, 1) != GEMMQ_OK || M == 0 || N == 0) return 0;
  const int64_t groups = act_grad_groups(type, M, N);
  return groups > 1 ? align_up(8 * groups * (int64_t)align_up(N, 4), 256) : 0;
}

int gemmq_act_grad(int act, int type, const void* Z, int64_t ldz, const void* U, int64_t ldu,
                   const void* dY, int64_t lddy, void* dZ, int64_t lddz, void* dU, int64_t lddu,
                   float* db, float* dbu, int64_t M, int64_t N, void* ws, size_t ws_bytes,
                   void* stream) {
  int rc = check_shape(M, N, 1);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type) || !known_act(act)) return GEMMQ_E_INVALID_ARG;
  // (a matrix without rows may have no address)
  if (M > 0 && (!U != !dU || (dbu && !U))) return GEMMQ_E_INVALID_ARG;
  if (db && db == dbu) return GEMMQ_E_INVALID_ARG;
  if (!aligned(db, 4) || !aligned(dbu, 4)) return GEMMQ_E_ALIGNMENT;
  const bool sums = db || dbu;
  if (N == 0 || (M == 0 && !sums)) return GEMMQ_OK;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (M > 0) {
    rc = check_rows(type, Z, ldz, N);
    if (rc == GEMMQ_OK) rc = check_rows(type, dY, lddy, N);
    if (rc == GEMMQ_OK) rc = check_rows(type, dZ, lddz, N);
    if (rc == GEMMQ_OK) rc = check_optional(type, U, ldu, N);
    if (rc == GEMMQ_OK) rc = check_optional(type, dU, lddu, N);
    if (rc != GEMMQ_OK) return rc;
    if (!same_rows(dZ, lddz, Z, ldz, M) || !same_rows(dZ, lddz, dY, lddy, M) ||
        !same_rows(dU, lddu, U, ldu, M) || !same_rows(dU, lddu, dY, lddy, M) || dZ == dU)
      return GEMMQ_E_INVALID_ARG;
    if (sums) rc = check_need(ws, ws_bytes, gemmq_act_grad_workspace(type, M, N));
  }
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  clear_pending();
  if (M == 0)  // sums of nothing
    return launched(launch_join({nullptr, db}, {nullptr, dbu}, 0, 0, (int)N, st));
  const int groups = act_grad_groups(type, M, N);
  const bool join = sums && groups > 1;  // else the kernel's sums are the results
  const int64_t np = (int64_t)align_up(N, 4);
  float* part = static_cast<float*>(ws);
  ActGradArgs a{rows(type, Z, ldz),   rows(type, U, ldu),   rows(type, dY, lddy),
                rows(type, dZ, lddz), rows(type, dU, lddu), {db, dbu}, np, act, type,
                (int)M, (int)N, 0};
  if (join) {
    a.sums[0] = db ? part : nullptr;
    a.sums[1] = dbu ? part + groups * np : nullptr;
  }
  rc = launched(launch_act_grad(a, st));
  if (rc != GEMMQ_OK || !join) return rc;
  return launched(launch_join({a.sums[0], db}, {a.sums[1], dbu}, np, groups, (int)N, st));
}

size_t gemmq_sample_workspace(int64_t M, int64_t N) {
  if (check_shape(M, N, 1) != GEMMQ_OK || M == 0 || N == 0) return 0;
  return sample_workspace(M, N);
}

int gemmq_sample(int type, const void* Z, int64_t ldz, const float* temperature,
                 const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                 int64_t* token, float* logprob, int64_t M, int64_t N, void* ws, size_t ws_bytes,
                 void* stream) {
  int rc = check_shape(M, N, 1);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type)) return GEMMQ_E_INVALID_ARG;
  if (N == 0) return GEMMQ_E_SHAPE;
  if (M == 0) return GEMMQ_OK;
  rc = check_rows(type, Z, ldz, N);
  if (rc != GEMMQ_OK) return rc;
  if (!u || !token) return GEMMQ_E_INVALID_ARG;
  if (!aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) || !aligned(min_p, 4) ||
      !aligned(u, 4) || !aligned(token, 8) || !aligned(logprob, 4))
    return GEMMQ_E_ALIGNMENT;
  rc = check_need(ws, ws_bytes, gemmq_sample_workspace(M, N));
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  SampleArgs a{};
  a.Z = Z;
  a.ldz = ldz;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.token = token;
  a.logprob = logprob;
  a.N = (int)N;
  a.wide = wide_rows(Z, ldz, type);
  clear_pending();
  return launched(launch_sample(a, type, M, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
