// i8_skinny.hip -- launches of the int8 product for few tokens (i8_skinny.h) for the
// linear layer, the vocabulary loss and its gradient's softmax factor.
#include "i8_skinny.h"

namespace gemmq {
namespace i8 {

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
  return launch_quantizing<kLinear>(a, xtype, X, ldx, st);
}

}  // namespace i8
}  // namespace gemmq
