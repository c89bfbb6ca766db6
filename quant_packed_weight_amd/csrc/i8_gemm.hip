// i8_gemm.hip -- the int8 product I[n, m] = sum_k W[n, k] X[m, k] on the matrix
// cores, with the three epilogues that read it: the scaled output of the linear
// layer, the softmax statistics of the vocabulary loss, and the softmax factor
// of its gradient.
//
// One workgroup computes a tile of BN channels by BM tokens, K in steps of 128
// bytes, both operands staged in LDS by direct buffer->LDS loads, two steps
// deep.  W is the MFMA's row operand, so a lane ends with one token and four
// consecutive channels per register quad: rows of Y are stored four values at a
// time, and the softmax sums of a token are in-lane sums.
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// LDS image of a step: rows of 128 bytes, eight 16-byte chunks each, chunk c of
// row r in slot c ^ (r & 7).  The eight rows that eight consecutive lanes read
// the same chunk of then lie in eight different slots, i.e. in different banks.
constexpr int kStep = 128;

enum Epilogue { kLinear, kLoss, kFactor };

struct TileArgs {
  Operands op;
  LinearOut lin;
  LossOut loss;
  FactorOut fac;
  uint32_t mtiles;
};

template <int BN, int BM>
struct Stage {
  static constexpr int kW = 0, kX = BN * kStep, kBytes = (BN + BM) * kStep;
};

// One operand's rows [row0, row0 + ROWS) of a step to LDS: instruction j of the
// workgroup's ROWS / 8 covers eight rows.  Rows past the matrix repeat its last
// row (their results are dropped), chunks past column K the row's last chunk (the
// activations are zeroed there, see clear_tail), so every access is inside.
template <int ROWS, int NW>
struct RowLoader {
  static constexpr int kIssues = ROWS / 8 / NW;
  static_assert(ROWS % (8 * NW) == 0, "every wave issues the same number of loads");
  rsrc_t rs;
  uint32_t voff[kIssues];
  int last;  // offset of the 16-byte chunk that holds column K - 1
  int chunk;

  __device__ __forceinline__ void init(const int8_t* base, int64_t ld, int64_t row0, int rows,
                                       int K, int wave, int lane) {
    const int valid = (int)min((int64_t)ROWS, rows - row0);
    rs = gk::make_rsrc(base + row0 * ld, (uint32_t)(valid * ld));
    chunk = 16 * ((lane & 7) ^ (lane >> 3));
    last = (K - 1) / 16 * 16;
#pragma unroll
    for (int j = 0; j < kIssues; ++j) {
      const int r = 8 * (wave + NW * j) + (lane >> 3);
      voff[j] = (uint32_t)(min(r, valid - 1) * ld) + chunk;
    }
  }
  __device__ __forceinline__ void issue(int k0, uint32_t lds, int wave) const {
    const int over = min(0, last - (k0 + chunk));  // <= 0, and chunk + over >= 0
#pragma unroll
    for (int j = 0; j < kIssues; ++j)
      gk::dma16(rs, voff[j] + (uint32_t)over, (uint32_t)k0, lds + 1024 * (wave + NW * j));
  }
};

__device__ __forceinline__ v4i frag(const uint8_t* tile, int row, int chunk) {
  return *reinterpret_cast<const v4i*>(tile + row * kStep + 16 * (chunk ^ (row & 7)));
}

// The activations' bytes from column K on, zeroed in LDS for the step at k0:
// whatever the rows' padding holds, and whatever W's holds, then adds nothing.
template <int BM, int THREADS>
__device__ __forceinline__ void clear_tail(uint8_t* x, int k0, int K, int t) {
  for (int i = t; i < BM * 8; i += THREADS) {
    const int row = i >> 3, c = i & 7, keep = K - (k0 + 16 * c);
    if (keep >= 16) continue;
    uint32_t* p = reinterpret_cast<uint32_t*>(x + row * kStep + 16 * (c ^ (row & 7)));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int b = keep - 4 * w;
      p[w] = b <= 0 ? 0u : b >= 4 ? p[w] : p[w] & ((1u << (8 * b)) - 1u);
    }
  }
}

template <int BN, int BM, int WN, int WM, int EPI>
__global__ __launch_bounds__(64 * WN * WM) void tile_kernel(TileArgs a) {
  constexpr int NW = WN * WM, T = 64 * NW;
  constexpr int TN = BN / WN / 32, TM = BM / WM / 32;
  using S = Stage<BN, BM>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * S::kBytes];
  __shared__ float swl[BN];
  __shared__ float2 red[EPI == kLoss ? WN * BM : 1];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = wave % WN, wm = wave / WN;
  const uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(id % a.mtiles) * BM, n0 = (int64_t)(id / a.mtiles) * BN;
  const Operands& op = a.op;

  RowLoader<BN, NW> lw;
  RowLoader<BM, NW> lx;
  lw.init(op.W, op.ldw, n0, op.N, op.K, wave, lane);
  lx.init(op.X, op.ldx, m0, op.M, op.K, wave, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;

  for (int i = t; i < BN; i += T) swl[i] = n0 + i < op.N ? op.sw[n0 + i] : 0.0f;

  v16i acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  const int steps = (op.K + kStep - 1) / kStep;
  lw.issue(0, lds0 + S::kW, wave);
  lx.issue(0, lds0 + S::kX, wave);
  for (int s = 0; s < steps; ++s) {
    uint8_t* cur = lds + (s & 1) * S::kBytes;
    gk::wait_vm<0>();
    gk::lds_barrier();  // this step is in LDS, and the other buffer is read
    if (s + 1 < steps) {
      const uint32_t nxt = lds0 + ((s + 1) & 1) * S::kBytes;
      lw.issue((s + 1) * kStep, nxt + S::kW, wave);
      lx.issue((s + 1) * kStep, nxt + S::kX, wave);
    } else if (op.K % kStep) {
      clear_tail<BM, T>(cur + S::kX, s * kStep, op.K, t);
      gk::lds_barrier();
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v4i wf[TN], xf[TM];
#pragma unroll
      for (int i = 0; i < TN; ++i)
        wf[i] = frag(cur + S::kW, (wn * TN + i) * 32 + (lane & 31), 2 * q + (lane >> 5));
#pragma unroll
      for (int j = 0; j < TM; ++j)
        xf[j] = frag(cur + S::kX, (wm * TM + j) * 32 + (lane & 31), 2 * q + (lane >> 5));
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = gk::mfma_i8(wf[i], xf[j], acc[i][j]);
    }
  }

  // Lane l holds token 32 (wm TM + j) + (l & 31) and, in registers 4 g .. 4 g + 3
  // of tile i, channels 32 (wn TN + i) + 8 g + 4 (l >> 5) + 0..3.
  const int h = lane >> 5;
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int ml = (wm * TM + j) * 32 + (lane & 31);
    const int64_t m = m0 + ml;
    const bool inside = m < op.M;
    const float sx = inside ? op.sx[m] : 0.0f;
    if constexpr (EPI == kLinear) {
      if (!inside) continue;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int nl = (wn * TN + i) * 32 + 8 * g + 4 * h;
          const int64_t n = n0 + nl;
          const int count = (int)min((int64_t)4, op.N - n);
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = (float)acc[i][j][4 * g + e] * sx * swl[nl + e];
            if (a.lin.bias && e < count) v[e] += a.lin.bias[n + e];
          }
          store4_as(a.lin.Y, m * a.lin.ldy + n, a.lin.type, a.lin.wide, count, v[0], v[1], v[2],
                    v[3]);
        }
    } else if constexpr (EPI == kLoss) {
      // base-2 logits: exp(z) = 2^(z log2 e), the factor folded into sx
      const float s2 = sx * kLog2e;
      const int64_t tg = inside ? a.loss.target[m] : -1;
      float top = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int nl = (wn * TN + i) * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
          const float z = (float)acc[i][j][r] * s2 * swl[nl];
          if (n0 + nl == tg) a.loss.zt[m] = z;
          // a NaN (a row whose scale is NaN) has to survive: it is not dropped by >
          if (n0 + nl < op.N) top = z > top || z != z ? z : top;
        }
      {
        const float o = __shfl_xor(top, 32, 64);
        top = o > top || o != o ? o : top;
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int nl = (wn * TN + i) * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
          const float z = (float)acc[i][j][r] * s2 * swl[nl];
          if (n0 + nl < op.N) sum += __builtin_amdgcn_exp2f(z - top);
        }
      sum += __shfl_xor(sum, 32, 64);
      if (h == 0) red[wn * BM + ml] = make_float2(top, sum);
    } else {
      const int64_t tg = inside ? a.fac.target[m] - a.fac.n0 : -1;
      const float s2 = sx * kLog2e, l2 = inside ? a.fac.lse[m] * kLog2e : 0.0f;
      if (!inside) continue;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int nl = (wn * TN + i) * 32 + 8 * g + 4 * h;
          if (n0 + nl >= a.fac.pitch) continue;  // the pitch is a multiple of 4
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float z = (float)acc[i][j][4 * g + e] * s2 * swl[nl + e];
            float p = __builtin_amdgcn_exp2f(z - l2);
            if (n0 + nl + e == tg) p -= 1.0f;
            v[e] = n0 + nl + e < op.N ? p * swl[nl + e] : 0.0f;
          }
          uint16_t* out = a.fac.P + m * a.fac.pitch + n0 + nl;
          for (int p = 0; p < a.fac.planes; ++p) {
            const bool last = p + 1 == a.fac.planes;
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = bf16_part(v[e], last);
            *reinterpret_cast<uint2*>(out + p * op.M * a.fac.pitch) =
                make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
          }
        }
    }
  }
  if constexpr (EPI == kLoss) {
    __syncthreads();
    for (int ml = t; ml < BM; ml += T) {
      if (m0 + ml >= op.M) break;
      float top = red[ml].x;
#pragma unroll
      for (int w = 1; w < WN; ++w) {
        const float o = red[w * BM + ml].x;
        top = o > top || o != o ? o : top;
      }
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float2 p = red[w * BM + ml];
        // a wave with no valid column has (-inf, 0)
        sum += p.y == 0.0f ? 0.0f : p.y * __builtin_amdgcn_exp2f(p.x - top);
      }
      a.loss.part[(m0 + ml) * a.loss.ntiles + n0 / BN] = make_float2(top, sum);
    }
  }
}

// The tiles of each row joined by log-sum-exp, one wave per row.
__global__ __launch_bounds__(256) void loss_join_kernel(LossOut o, float* loss, float* lse, int M,
                                                        int64_t N) {
  const int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= M) return;
  const float2* p = o.part + m * o.ntiles;
  float top = -__builtin_inff();
  for (int i = lane; i < o.ntiles; i += 64) {
    const float z = p[i].x;
    top = z > top || z != z ? z : top;
  }
  for (int d = 1; d < 64; d *= 2) {
    const float z = __shfl_xor(top, d, 64);
    top = z > top || z != z ? z : top;
  }
  float sum = 0.0f;
  for (int i = lane; i < o.ntiles; i += 64) sum += p[i].y * __builtin_amdgcn_exp2f(p[i].x - top);
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d, 64);
  if (lane == 0) {
    const float l2 = top + __builtin_log2f(sum);
    const int64_t tg = o.target[m];
    lse[m] = l2 * kLn2;
    loss[m] = tg < 0 ? 0.0f : tg >= N ? __builtin_nanf("") : (l2 - o.zt[m]) * kLn2;
  }
}

constexpr int kBN = 128;
constexpr int64_t kMaxGrid = 0x7fffffff;

int64_t tiles(int M, int N, int bm) { return ceil_div(M, bm) * ceil_div(N, kBN); }
int pick_bm(int M) { return M <= 32 ? 32 : 128; }

template <int EPI>
int launch_tiles(TileArgs& a, hipStream_t st) {
  const int bm = pick_bm(a.op.M);
  const int64_t n = tiles(a.op.M, a.op.N, bm);
  if (n > kMaxGrid) return -1;
  a.mtiles = (uint32_t)ceil_div(a.op.M, bm);
  if (bm == 32)
    tile_kernel<kBN, 32, 4, 1, EPI><<<(uint32_t)n, 256, 0, st>>>(a);
  else
    tile_kernel<kBN, 128, 2, 2, EPI><<<(uint32_t)n, 256, 0, st>>>(a);
  return 0;
}

}  // namespace

bool linear_fits(int M, int N) { return tiles(M, N, pick_bm(M)) <= kMaxGrid; }
bool loss_fits(int M, int N, int) { return linear_fits(M, N); }
bool factor_fits(int M, int N) { return linear_fits(M, N); }

int launch_linear(const Operands& op, const LinearOut& out, hipStream_t st) {
  TileArgs a{};
  a.op = op;
  a.lin = out;
  return launch_tiles<kLinear>(a, st);
}

int loss_tiles(int, int N, int) { return (int)ceil_div(N, kBN); }

int launch_loss(const Operands& op, const LossOut& out, hipStream_t st) {
  TileArgs a{};
  a.op = op;
  a.loss = out;
  return launch_tiles<kLoss>(a, st);
}

int launch_loss_join(const LossOut& o, float* loss, float* lse, int M, int N, hipStream_t st) {
  loss_join_kernel<<<(uint32_t)ceil_div(M, 4), 256, 0, st>>>(o, loss, lse, M, N);
  return 0;
}

int launch_factor(const Operands& op, const FactorOut& out, hipStream_t st) {
  TileArgs a{};
  a.op = op;
  a.fac = out;
  return launch_tiles<kFactor>(a, st);
}

}  // namespace i8
}  // namespace gemmq
