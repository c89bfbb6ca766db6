// i8_act.hip -- launches of the int8 product whose epilogue has an activation and a
// residual, and of the gated pair of products: the kernels of i8_tile.h and i8_skinny.h,
// by the same choices.  A pair counts as a product of 2 N rows.
#include "i8_skinny.h"
#include "i8_tile.h"

namespace gemmq {
namespace i8 {
namespace {

int rows_of(int N, bool pair) { return pair ? 2 * N : N; }

}  // namespace

bool act_fits(int M, int N, int K, bool pair) { return product_fits(M, rows_of(N, pair), K); }

int launch_act(const Operands& op, const ActOut& out, bool pair, hipStream_t st) {
  if (skinny(op.M, rows_of(op.N, pair), true)) {
    SkinnyArgs a{};
    a.op = op;
    a.act = out;
    return pair ? launch<kGate>(a, st) : launch<kAct>(a, st);
  }
  TileArgs a{};
  a.op = op;
  a.act = out;
  return pair ? launch_tiles<kGate>(a, st) : launch_tiles<kAct>(a, st);
}

bool act_fuses(int M, int N, int K, bool pair) { return fuses(M, rows_of(N, pair), K); }

int launch_act_fused(int xtype, const void* X, int64_t ldx, const Operands& op, const ActOut& out,
                     bool pair, hipStream_t st) {
  SkinnyArgs a{};
  a.op = op;
  a.act = out;
  return pair ? launch_quantizing<kGate>(a, xtype, X, ldx, st)
              : launch_quantizing<kAct>(a, xtype, X, ldx, st);
}

}  // namespace i8
}  // namespace gemmq
