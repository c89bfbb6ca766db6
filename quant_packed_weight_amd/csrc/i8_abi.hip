// i8_abi.hip -- the int8 half of the C ABI (gemmq_i8.h): validation, workspace
// layout and the order of launches.  As in abi.hip, a bad call returns a named
// status and launches nothing, and the library owns no memory.
#include "i8_check.h"

using gemmq::aligned;
using gemmq::check_device;
using gemmq::clear_pending;
using gemmq::launched;
using namespace gemmq::i8;

namespace {

// The gradients walk N in pieces whose bf16 factor stays within this many bytes, or
// of kMinPiece columns where the rows alone are more: it bounds the workspace.  A
// further piece costs a passage of the partial sums through memory and another
// last round of tiles, more than a factor that fits the 256 MB last-level cache
// saves (bf16 over 151936 x 2048, with 128 / 256 / 384 / 768 MB: M = 1024 1028 / 956 /
// 913 / 913 us, one piece from 384; M = 2048 1881 / 1858 / 1800 / 1735; f32 at M = 700
// 1578 / 1618 / 1568 / 1539).  768 MB would buy 4% there with twice the memory.
constexpr int64_t kFactorBytes = (int64_t)384 << 20;
constexpr int64_t kMinPiece = 1024;

// Up to eight rows of bf16 have two numbers for each value of the factor, in the
// workspace or, where dY is read as it lies, in the product's LDS: one's rounding errors
// have the fewest rows to even out in, and the product waits for W more than for the
// matrix cores.
int grad_planes(int type, int64_t M) { return type == GEMMQ_BF16 && M <= 8 ? 2 : planes_of(type); }

struct GradPlan {
  int planes;
  GradSplit split;
  int64_t piece, kp;
  bool direct;  // one piece and one range: no partial sums
  size_t factor_bytes, acc_bytes;
  size_t bytes() const { return factor_bytes + acc_bytes; }
};

GradPlan grad_plan(int planes, int64_t M, int64_t N, int64_t K) {
  GradPlan p;
  p.planes = planes;
  int64_t most = kFactorBytes / (2 * p.planes * M) / 256 * 256;
  if (most < kMinPiece) most = kMinPiece;
  const int64_t n64 = (int64_t)align_up(N < 1 ? 1 : N, 64);
  // equal pieces, in multiples of 256 columns
  const int64_t pieces = ceil_div(n64, most);
  p.piece = pieces == 1 ? n64 : (int64_t)align_up(ceil_div(n64, pieces), 256);
  p.kp = (int64_t)align_up(K, 4);
  p.split = grad_split((int)M, (int)p.piece, (int)K, p.planes, pieces == 1);
  p.direct = pieces == 1 && p.split.splits == 1;
  p.factor_bytes = align_up(2 * p.planes * M * p.piece, 256);
  p.acc_bytes = p.direct ? 0 : align_up(4 * p.split.splits * M * p.kp, 256);
  return p;
}

bool grad_shape_ok(int64_t M, int64_t K, const GradPlan& p) {
  return grad_fits(p.split, (int)M, (int)K) && product_fits((int)M, (int)p.piece, (int)K);
}

// Up to 128 tokens a bf16 dY whose rows allow 16-byte loads is read by the product as
// it lies, and W scaled by sw instead (a rounding of sw * w to bf16 in the place of one
// of dy * sw; up to eight tokens dY is scaled, in two numbers): no factor in the
// workspace, and a launch less (4096 x 4096 at M = 16 15 -> 12 us, M = 128 29 -> 26).
// With more tokens the large tiles are the faster ones, whose conversion has no room for
// the scaling: with the factor / as it lies M = 129 over 2048 x 2048 15.4 / 14.3 us, 4096
// x 12288 39 / 50, M = 512 68 / 82.
constexpr int64_t kScaledMaxM = 128;

bool reads_dy(int type, const void* dY, int64_t lddy, int64_t M, int64_t N) {
  return type == GEMMQ_BF16 && M <= kScaledMaxM && N % 8 == 0 && N > 0 &&
         wide_rows(dY, lddy, type) && lddy <= ((int64_t)1 << 22);
}

GradPlan direct_plan(int64_t M, int64_t N, int64_t K) {
  GradPlan p;
  p.planes = grad_planes(GEMMQ_BF16, M);
  p.piece = N;
  p.kp = (int64_t)align_up(K, 4);
  p.split = grad_split((int)M, (int)N, (int)K, p.planes, true);
  p.direct = p.split.splits == 1;
  p.factor_bytes = 0;
  p.acc_bytes = p.direct ? 0 : align_up(4 * p.split.splits * M * p.kp, 256);
  return p;
}

// The pieces of a gradient: `factor` enqueues the factor of columns [n0, n0 + n)
// at a pitch into the workspace, and the product with W's rows follows it.
template <class Factor>
int run_grad(const GradPlan& p, const int8_t* W, int64_t ldw, const GradOut& out, int64_t M,
             int64_t N, int64_t K, void* ws, hipStream_t st, Factor factor) {
  uint16_t* P = static_cast<uint16_t*>(ws);
  float* acc = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.factor_bytes);
  clear_pending();
  for (int64_t n0 = 0; n0 < N; n0 += p.piece) {
    const int64_t n = N - n0 < p.piece ? N - n0 : p.piece;
    const int64_t pitch = (int64_t)align_up(n, 64);
    int rc = launched(factor(n0, n, P, pitch));
    if (rc != GEMMQ_OK) return rc;
    const GradArgs g{W + n0 * ldw, ldw,      P,
                     pitch,        p.direct ? nullptr : acc, p.kp,
                     (int)M,       (int)n,   (int)K,
                     p.planes,     p.split.tile, p.split.splits,
                     n0 > 0,       nullptr, out};
    rc = launched(launch_grad(g, st));
    if (rc != GEMMQ_OK) return rc;
  }
  if (p.direct && N > 0) return GEMMQ_OK;
  return launched(
      launch_finish(acc, p.kp, N > 0 ? p.split.splits : 0, out, (int)M, (int)K, st));
}

// The loss's factor is often a few large numbers a row: exp(z - lse) - 1 at the target,
// and exp(z - lse) of the likeliest others.  With one bf16 number each their few
// roundings do not average out (M = 2 over 3137 x 768 2.8e-3 relative, the result's
// own rounding 1.6e-3).  So what is left of the target's is kept, and added at the end
// (2.3e-3), and see grad_planes.
size_t rest_bytes(const GradPlan& p, int64_t M) { return p.planes == 1 ? align_up(4 * M, 256) : 0; }

GradOut grad_out(int type, void* dX, int64_t lddx) {
  GradOut o{};
  o.type = type;
  o.dX = dX;
  o.lddx = lddx;
  o.wide = lddx % 4 == 0 && aligned(dX, (uintptr_t)(4 * type_bytes(type)));
  return o;
}

}  // namespace

extern "C" {

int gemmq_i8_abi_version(void) { return GEMMQ_I8_ABI_VERSION; }

int gemmq_quantize_i8(int xtype, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* s,
                      int64_t M, int64_t K, void* stream) {
  int rc = check_shape(M, 0, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(xtype)) return GEMMQ_E_INVALID_ARG;
  if (M == 0) return GEMMQ_OK;
  rc = check_rows(xtype, X, ldx, K);
  if (rc == GEMMQ_OK) rc = check_i8(Q, ldq, s, K);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  clear_pending();
  return launched(launch_quantize(xtype, X, ldx, Q, ldq, s, (int)M, (int)K,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// the product's own checks and its argument blocks
int check_product(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Xq, int64_t ldq,
                  const float* sx, const float* bias, int ytype, void* Y, int64_t ldy, int64_t M,
                  int64_t N, int64_t K, Operands& op, LinearOut& out) {
  int rc = check_i8(W, ldw, sw, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc == GEMMQ_OK) rc = check_rows(ytype, Y, ldy, N);
  if (rc != GEMMQ_OK) return rc;
  if (bias && !aligned(bias, 4)) return GEMMQ_E_ALIGNMENT;
  if (!product_fits((int)M, (int)N, (int)K)) return GEMMQ_E_SHAPE;
  op = Operands{W, sw, Xq, sx, ldw, ldq, (int)M, (int)N, (int)K};
  out = LinearOut{bias, Y, ldy, ytype,
                  ldy % 4 == 0 && aligned(Y, (uintptr_t)(4 * type_bytes(ytype))),
                  type_bytes(ytype) == 2 && wide_rows(Y, ldy, ytype)};
  return GEMMQ_OK;
}

}  // namespace

extern "C" {

int gemmq_gemm_i8(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Xq, int64_t ldq,
                  const float* sx, const float* bias, int ytype, void* Y, int64_t ldy, int64_t M,
                  int64_t N, int64_t K, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(ytype)) return GEMMQ_E_INVALID_ARG;
  if (M == 0 || N == 0) return GEMMQ_OK;
  Operands op;
  LinearOut out;
  rc = check_product(W, ldw, sw, Xq, ldq, sx, bias, ytype, Y, ldy, M, N, K, op, out);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  clear_pending();
  return launched(launch_linear(op, out, static_cast<hipStream_t>(stream)));
}

int gemmq_linear_i8(const int8_t* W, int64_t ldw, const float* sw, int xtype, const void* X,
                    int64_t ldx, int8_t* Xq, int64_t ldq, float* sx, const float* bias, int ytype,
                    void* Y, int64_t ldy, int64_t M, int64_t N, int64_t K, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(xtype) || !known(ytype)) return GEMMQ_E_INVALID_ARG;
  if (M == 0) return GEMMQ_OK;
  rc = check_rows(xtype, X, ldx, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc != GEMMQ_OK) return rc;
  Operands op;
  LinearOut out;
  if (N > 0) rc = check_product(W, ldw, sw, Xq, ldq, sx, bias, ytype, Y, ldy, M, N, K, op, out);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  clear_pending();
  if (N > 0 && fuses((int)M, (int)N, (int)K) &&
      !share_memory(span(xtype, X, ldx, K), span(ytype, Y, ldy, N), M))
    return launched(launch_fused(xtype, X, ldx, op, out, st));
  rc = launched(launch_quantize(xtype, X, ldx, Xq, ldq, sx, (int)M, (int)K, st));
  if (rc != GEMMQ_OK || N == 0) return rc;
  return launched(launch_linear(op, out, st));
}

size_t gemmq_linear_i8_grad_workspace(int type, int64_t M, int64_t N, int64_t K) {
  if (!known(type) || check_shape(M, N, K) != GEMMQ_OK || M == 0) return 0;
  const GradPlan p = grad_plan(grad_planes(type, M), M, N, K);
  if (!grad_shape_ok(M, K, p)) return 0;
  // whichever way dY's rows will allow
  if (type != GEMMQ_BF16 || N == 0 || M > kScaledMaxM) return p.bytes();
  const GradPlan d = direct_plan(M, N, K);
  if (!grad_fits(d.split, (int)M, (int)K)) return 0;
  return d.bytes() > p.bytes() ? d.bytes() : p.bytes();
}

int gemmq_linear_i8_grad(const int8_t* W, int64_t ldw, const float* sw, int type, const void* dY,
                         int64_t lddy, void* dX, int64_t lddx, int64_t M, int64_t N, int64_t K,
                         void* ws, size_t ws_bytes, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type)) return GEMMQ_E_INVALID_ARG;
  if (M == 0) return GEMMQ_OK;
  rc = check_rows(type, dX, lddx, K);
  if (rc == GEMMQ_OK && N > 0) rc = check_i8(W, ldw, sw, K);
  if (rc == GEMMQ_OK && N > 0) rc = check_rows(type, dY, lddy, N);
  if (rc != GEMMQ_OK) return rc;
  const GradPlan p = grad_plan(grad_planes(type, M), M, N, K);
  const size_t need = gemmq_linear_i8_grad_workspace(type, M, N, K);
  if (need == 0) return GEMMQ_E_SHAPE;
  rc = check_ws(ws, ws_bytes, need);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (reads_dy(type, dY, lddy, M, N)) {
    const GradPlan d = direct_plan(M, N, K);
    const GradOut out = grad_out(type, dX, lddx);
    float* acc = d.direct ? nullptr : static_cast<float*>(ws);
    const GradArgs g{W,         ldw,
                     static_cast<const uint16_t*>(dY), lddy,
                     acc,       d.kp,
                     (int)M,    (int)N,
                     (int)K,    d.planes,
                     d.split.tile, d.split.splits,
                     false,     sw,
                     out};
    clear_pending();
    rc = launched(launch_grad(g, st));
    if (rc != GEMMQ_OK || d.direct) return rc;
    return launched(launch_finish(acc, d.kp, d.split.splits, out, (int)M, (int)K, st));
  }
  return run_grad(p, W, ldw, grad_out(type, dX, lddx), M, N, K, ws, st,
                  [&](int64_t n0, int64_t n, uint16_t* P, int64_t pitch) {
                    const uint8_t* dy = static_cast<const uint8_t*>(dY) + n0 * type_bytes(type);
                    return launch_planes(type, dy, lddy, sw + n0, P, pitch, p.planes, (int)M,
                                         (int)n, st);
                  });
}

size_t gemmq_loss_i8_workspace(int64_t M, int64_t N, int64_t K) {
  if (check_shape(M, N, K) != GEMMQ_OK || M == 0 || N == 0 || !product_fits((int)M, (int)N, (int)K))
    return 0;
  return align_up(8 * M * loss_tiles((int)M, (int)N, (int)K), 256);
}

int gemmq_loss_i8(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Xq, int64_t ldq,
                  const float* sx, const int64_t* target, float* loss, float* lse, int64_t M,
                  int64_t N, int64_t K, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (N == 0) return GEMMQ_E_SHAPE;
  if (M == 0) return GEMMQ_OK;
  rc = check_i8(W, ldw, sw, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc != GEMMQ_OK) return rc;
  if (!target || !loss || !lse) return GEMMQ_E_INVALID_ARG;
  if (!aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4)) return GEMMQ_E_ALIGNMENT;
  const size_t need = gemmq_loss_i8_workspace(M, N, K);
  if (need == 0) return GEMMQ_E_SHAPE;
  rc = check_ws(ws, ws_bytes, need);
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  const Operands op{W, sw, Xq, sx, ldw, ldq, (int)M, (int)N, (int)K};
  const int nt = loss_tiles((int)M, (int)N, (int)K);
  const LossOut o{target, static_cast<float2*>(ws), nt};
  hipStream_t st = static_cast<hipStream_t>(stream);
  clear_pending();
  rc = launched(launch_loss(op, o, st));
  if (rc != GEMMQ_OK) return rc;
  return launched(launch_loss_join(op, o, loss, lse, st));
}

size_t gemmq_loss_i8_grad_workspace(int type, int64_t M, int64_t N, int64_t K) {
  if (!known(type) || check_shape(M, N, K) != GEMMQ_OK || M == 0 || N == 0) return 0;
  const GradPlan p = grad_plan(grad_planes(type, M), M, N, K);
  return grad_shape_ok(M, K, p) ? p.bytes() + rest_bytes(p, M) : 0;
}

int gemmq_loss_i8_grad(const int8_t* W, int64_t ldw, const float* sw, const int8_t* Xq,
                       int64_t ldq, const float* sx, const int64_t* target, const float* lse,
                       const float* dloss, int type, void* dX, int64_t lddx, int64_t M, int64_t N,
                       int64_t K, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_shape(M, N, K);
  if (rc != GEMMQ_OK) return rc;
  if (!known(type)) return GEMMQ_E_INVALID_ARG;
  if (N == 0) return GEMMQ_E_SHAPE;
  if (M == 0) return GEMMQ_OK;
  rc = check_i8(W, ldw, sw, K);
  if (rc == GEMMQ_OK) rc = check_i8(Xq, ldq, sx, K);
  if (rc == GEMMQ_OK) rc = check_rows(type, dX, lddx, K);
  if (rc != GEMMQ_OK) return rc;
  if (!target || !lse || !dloss) return GEMMQ_E_INVALID_ARG;
  if (!aligned(target, 8) || !aligned(lse, 4) || !aligned(dloss, 4)) return GEMMQ_E_ALIGNMENT;
  const GradPlan p = grad_plan(grad_planes(type, M), M, N, K);
  if (!grad_shape_ok(M, K, p)) return GEMMQ_E_SHAPE;
  rc = check_ws(ws, ws_bytes, p.bytes() + rest_bytes(p, M));
  if (rc == GEMMQ_OK) rc = check_device();
  if (rc != GEMMQ_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  GradOut out = grad_out(type, dX, lddx);
  out.g = dloss;
  out.target = target;
  out.nvocab = N;
  float* rest = nullptr;
  if (rest_bytes(p, M)) {
    rest = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.bytes());
    out.rest = rest;
    out.W = W;
    out.ldw = ldw;
  }
  return run_grad(p, W, ldw, out, M, N, K, ws, st,
                  [&](int64_t n0, int64_t n, uint16_t* P, int64_t pitch) {
                    const Operands op{W + n0 * ldw, sw + n0, Xq,     sx,    ldw,
                                      ldq,          (int)M,  (int)n, (int)K};
                    const FactorOut f{target, lse, P, pitch, n0, p.planes, rest};
                    return launch_factor(op, f, st);
                  });
}

}  // extern "C"
