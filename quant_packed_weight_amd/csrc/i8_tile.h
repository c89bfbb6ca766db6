// i8_tile.h -- the int8 product I[n, m] = sum_k W[n, k] X[m, k] on the matrix cores by
// tiles in LDS: the kernel, with the epilogues that read the sums (the scaled output of
// the linear layer, the softmax statistics of the vocabulary loss and the softmax factor of
// its gradient, launched by i8_gemm.hip; an activation with a residual and the gated pair,
// launched by i8_act.hip), and the choice of the tile.
//
// One workgroup computes a tile of BN channels by BM tokens, K in steps of 128
// bytes, both operands staged in LDS by direct buffer->LDS loads.  W is the
// MFMA's row operand, so a lane ends with one token and four consecutive channels
// per register quad: rows of Y are stored four values at a time, and the softmax
// sums of a token are in-lane sums.
#pragma once

#include "i8_act.h"
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

// LDS image of a step: rows of 128 bytes, eight 16-byte chunks each, chunk c of
// row r in slot c ^ ((r >> 1) & 7).  Sixteen rows whose numbers differ in their
// low four bits then have the same chunk in sixteen different 16-byte columns of
// the 256 bytes that the 64 banks span: no conflict among sixteen lanes of a
// fragment's read (with c ^ (r & 7), eight columns, the reads took twice as long).
constexpr int kStep = 128;

__device__ __forceinline__ int slot(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

struct TileArgs {
  Operands op;
  LinearOut lin;
  LossOut loss;
  FactorOut fac;
  ActOut act;
  uint32_t mtiles, ntiles, group;
};

// the image of a tile of 16-bit results in LDS: CH / 8 chunks of 16 bytes a row, chunk c
// of row m in slot c ^ (m mod the largest power of two that divides CH / 8, or 8)
template <int CH>
struct Image {
  static constexpr int kChunks = CH / 8;
  static constexpr int kMix =
      (kChunks & (kChunks - 1)) == 0 ? kChunks - 1 : kChunks % 8 == 0 ? 7 : 3;
  static_assert(kChunks % 4 == 0, "the slots of a row are its own");
  static __device__ __forceinline__ int at(int row, int chunk) {
    return (row * kChunks + (chunk ^ (row & kMix))) * 16;
  }
};

// rows m0 .. of results [M, N] from column n0: between memory and their image (T threads,
// BM rows).  STORE: from the image; else to it, zero where there is nothing.  The stores are a
// stream's: what the L2 holds of the operands matters more to the tiles that follow (a pair of
// 2 x 12288 over 4096 with z and u kept, us: 128 tokens 33.7 -> 30.5, 2048 220 -> 215.5, 8192 856
// -> 838; with the next product 65 -> 62, 352 -> 343, 1277 -> 1240).
template <int CH, int BM, int T, bool STORE>
__device__ __forceinline__ void move_image(uint8_t* image, const Rows& rows, int64_t m0, int64_t n0,
                                           int M, int N, int t) {
  using I = Image<CH>;
  uint16_t* p = static_cast<uint16_t*>(rows.p);
  if (rows.lines) {
    for (int i = t; i < BM * I::kChunks; i += T) {
      const int ml = i / I::kChunks, c = i % I::kChunks;
      const int64_t n = n0 + 8 * c;
      if (m0 + ml >= M || n >= N) continue;
      v4i* in = reinterpret_cast<v4i*>(image + I::at(ml, c));
      uint16_t* to = p + (m0 + ml) * rows.ld + n;
      if (n + 8 <= N) {
        if constexpr (STORE)
          __builtin_nontemporal_store(*in, reinterpret_cast<v4i*>(to));
        else
          *in = *reinterpret_cast<const v4i*>(to);
      } else if constexpr (STORE) {
        const v4i v = *in;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < N) to[e] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
      } else {
        v4i v = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < N) v[e >> 1] |= (int)((uint32_t)to[e] << (16 * (e & 1)));
        *in = v;
      }
    }
  } else {
    // rows off 16 bytes: neighbouring lanes still access neighbouring values
    for (int i = t; i < BM * CH; i += T) {
      const int ml = i / CH, nl = i % CH;
      if (m0 + ml >= M || n0 + nl >= N) continue;
      uint16_t* in = reinterpret_cast<uint16_t*>(image + I::at(ml, nl >> 3) + 2 * (nl & 7));
      uint16_t* to = p + (m0 + ml) * rows.ld + n0 + nl;
      if constexpr (STORE)
        *to = *in;
      else
        *in = *to;
    }
  }
}

// Work list order: `group` tiles along the tokens by all tiles along the channels,
// then the next group.  The tiles that one XCD works on at a time are then about
// as many tokens as channels, and its L2 loads the fewest rows for them.
__device__ __forceinline__ void tile_of(const TileArgs& a, uint32_t id, uint32_t& tm,
                                        uint32_t& tn) {
  const uint32_t full = a.group * a.ntiles, g = id / full, r = id % full;
  const uint32_t width = min(a.group, a.mtiles - g * a.group);
  tm = g * a.group + r % width;
  tn = r / width;
}

template <int BN, int BM>
struct Stage {
  static constexpr int kW = 0, kX = BN * kStep, kBytes = (BN + BM) * kStep;
};

// One operand's rows [row0, row0 + ROWS) of a step to LDS: instruction j of the
// workgroup's ROWS / 8 covers eight rows.  Rows past the matrix repeat its last
// row (their results are dropped), chunks past column K the row's last chunk (the
// activations are zeroed there, see clear_tail), so every access is inside.
// PAIR: groups of eight rows alternate between two matrices' rows; a wave's are all of
// one of them.
template <int ROWS, int NW, bool PAIR = false>
struct RowLoader {
  static constexpr int kIssues = ROWS / 8 / NW;
  static_assert(ROWS % (8 * NW) == 0 && NW % 2 == 0, "each wave issues the same loads");
  rsrc_t rs;
  uint32_t voff[kIssues];
  int last;  // offset of the 16-byte chunk that holds column K - 1
  int chunk;

  __device__ __forceinline__ void init(const int8_t* base, int64_t ld, int64_t row0, int rows,
                                       int K, int wave, int lane) {
    const int valid = (int)min((int64_t)(PAIR ? ROWS / 2 : ROWS), rows - row0);
    rs = gk::make_rsrc(base + row0 * ld, (uint32_t)(valid * ld));
    // the eight rows of an instruction start at a multiple of eight, of sixteen
    // for even waves (NW is even): the slot of a lane's chunk is the same in all
    chunk = 16 * slot(8 * (wave & 1) + (lane >> 3), lane & 7);
    last = (K - 1) / 16 * 16;
#pragma unroll
    for (int j = 0; j < kIssues; ++j) {
      const int r = 8 * (PAIR ? (wave + NW * j) >> 1 : wave + NW * j) + (lane >> 3);
      voff[j] = (uint32_t)(min(r, valid - 1) * ld) + chunk;
    }
  }
  // how far the chunk of the step at column k0 moves back to lie before column K
  // (<= 0, and chunk + over >= 0)
  __device__ __forceinline__ uint32_t over(int k0) const {
    return (uint32_t)min(0, last - (k0 + chunk));
  }
  // load j, where the wave-uniform `take` is not zero
  __device__ __forceinline__ void issue(int j, uint32_t take, int k0, uint32_t back, uint32_t lds,
                                        int wave) const {
    gk::dma16_if(take, rs, voff[j] + back, (uint32_t)k0, lds + 1024 * (wave + NW * j));
  }
};

__device__ __forceinline__ v4i frag(const uint8_t* tile, int row, int chunk) {
  return *reinterpret_cast<const v4i*>(tile + row * kStep + 16 * slot(row, chunk));
}

// The activations' bytes from column K on, zeroed in LDS for the step at k0:
// whatever the rows' padding holds, and whatever W's holds, then adds nothing.
template <int BM, int THREADS>
__device__ __forceinline__ void clear_tail(uint8_t* x, int k0, int K, int t) {
  for (int i = t; i < BM * 8; i += THREADS) {
    const int row = i >> 3, c = i & 7, keep = K - (k0 + 16 * c);
    if (keep >= 16) continue;
    v4i* p = reinterpret_cast<v4i*>(x + row * kStep + 16 * slot(row, c));
    *p = keep <= 0 ? (v4i){0, 0, 0, 0} : keep_bytes(*p, keep);
  }
}

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
// the upper half of the wave's lanes in a and the lower half in b, exchanged
__device__ __forceinline__ v2u swap_halves(uint32_t a, uint32_t b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  return (v2u){r[0], r[1]};
}

// (max, sum) of one part of a row, the sum taken relative to the row's maximum; s2 as
// where the parts were made
__device__ __forceinline__ float join_term(float2 p, float top, float s2) {
  // a part without columns is (-inf, 0)
  return p.y == 0.0f ? 0.0f : p.y * __builtin_amdgcn_exp2f((p.x - top) * s2);
}

// The epilogues kAct and kGate of a tile's sums: y = act(z) + r, or act(z) u, and z and u
// where they are asked for, one after the other from the sums.  16-bit rows pass through
// their image in LDS (nothing else uses its bytes any more), the residual's on the same
// way and in the same place: each value is read and written by its lane in between, so
// the residual and the result may be one matrix.
template <int BN, int BM, int WN, int WM, int T, int EPI>
__device__ __forceinline__ void finish_act(const TileArgs& a, const v16i (&acc)[BN / WN / 32][BM / WM / 32],
                                           const float* swl, const float* bias, uint8_t* lds,
                                           int64_t m0, int64_t n0, int wn, int wm, int lane,
                                           int group, int t) {
  constexpr int TN = BN / WN / 32, TM = BM / WM / 32, CH = EPI == kGate ? BN / 2 : BN;
  const Operands& op = a.op;
  const int h = lane >> 5, nw = wn * TN * 32 + 4 * h;
  const bool edge = n0 + CH > op.N;
  const Act act = act_of(a.act.act);
  const int type = a.act.type;
  const bool wide16 = type != GEMMQ_F32;  // through LDS, as below
  if (wide16 && EPI == kAct && a.act.R.p) {
    move_image<CH, BM, T, false>(lds, a.act.R, m0, n0, op.M, op.N, t);
    __syncthreads();
  }
  // what: 0 the result, 1 and 2 the products before the activation
  auto emit = [&](int what, const Rows& rows) {
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      if (group > 0) break;
      const int ml = (wm * TM + j) * 32 + (lane & 31);
      const int64_t m = m0 + ml;
      if (m >= op.M) continue;
      const float sx = op.sx[m];
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        // four channels of registers 4 g .. 4 g + 3
        auto scaled4 = [&](int g, float(&v)[4]) {
          const int row = nw + 32 * i + 8 * g;
          const float4 sw = *reinterpret_cast<const float4*>(swl + row);
          const float4 b = *reinterpret_cast<const float4*>(bias + row);
          const v16i& c = acc[i][j];
          v[0] = fmaf((float)c[4 * g] * sx, sw.x, b.x);
          v[1] = fmaf((float)c[4 * g + 1] * sx, sw.y, b.y);
          v[2] = fmaf((float)c[4 * g + 2] * sx, sw.z, b.z);
          v[3] = fmaf((float)c[4 * g + 3] * sx, sw.w, b.w);
        };
#pragma unroll
        for (int g = 0; g < 4; g += EPI == kGate ? 2 : 1) {
          const int nl = EPI == kGate ? 16 * (wn * TN + i) + 4 * g + 4 * h : nw + 32 * i + 8 * g;
          const int64_t n = n0 + nl;
          const int count = edge ? (int)min((int64_t)4, op.N - n) : 4;
          uint2* in = reinterpret_cast<uint2*>(lds + Image<CH>::at(ml, nl >> 3) + 8 * h);
          float v[4];
          scaled4(EPI == kGate && what == 2 ? g + 1 : g, v);
          if (what == 0) {
            activate(act, v);
            float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (EPI == kGate) {
              scaled4(g + 1, o);
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] *= o[e];
            } else if (a.act.R.p) {
              if (wide16) {
                const uint2 r = *in;
                const float2 lo = halves(r.x, type), hi = halves(r.y, type);
                o[0] = lo.x, o[1] = lo.y, o[2] = hi.x, o[3] = hi.y;
              } else {
                load4_as(a.act.R.p, m * a.act.R.ld + n, type, a.act.R.wide, count, o);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += o[e];
            }
          }
          if (wide16)
            *in = make_uint2(two_bits(v[0], v[1], type), two_bits(v[2], v[3], type));
          else
            store4_as(rows.p, m * rows.ld + n, type, rows.wide, count, v[0], v[1], v[2], v[3]);
        }
      }
    }
    if (wide16) {
      __syncthreads();
      move_image<CH, BM, T, true>(lds, rows, m0, n0, op.M, op.N, t);
    }
  };
  emit(0, a.act.Y);
  if (a.act.Z.p) {
    if (wide16) __syncthreads();
    emit(1, a.act.Z);
  }
  if (EPI == kGate && a.act.U.p) {
    if (wide16) __syncthreads();
    emit(2, a.act.U);
  }
}

// GROUPS groups of WN x WM waves compute the tile, group g the steps g, g + GROUPS,
// ... of K in buffers of its own; their sums are added at the end.  More than one
// where the tiles leave the chip idle: a step is then mostly a round trip to LDS
// and back, and the groups' overlap.
template <int BN, int BM, int WN, int WM, int DEPTH, int GROUPS, int EPI>
__global__ __launch_bounds__(64 * WN * WM * GROUPS, 2) void tile_kernel(TileArgs a) {
  constexpr int NW = WN * WM, T = 64 * NW * GROUPS;
  constexpr int TN = BN / WN / 32, TM = BM / WM / 32;
  using S = Stage<BN, BM>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[GROUPS * DEPTH * S::kBytes];
  __shared__ __attribute__((aligned(16))) float swl[BN];
  constexpr bool kBiased = EPI == kLinear || EPI == kAct || EPI == kGate;
  constexpr int CH = EPI == kGate ? BN / 2 : BN;  // channels of the results
  __shared__ __attribute__((aligned(16))) float bias[kBiased ? BN : 4];
  __shared__ float2 red[EPI == kLoss ? WN * BM : 1];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane((t >> 6) % NW);
  const int group = GROUPS == 1 ? 0 : __builtin_amdgcn_readfirstlane((t >> 6) / NW);
  const int wn = wave % WN, wm = wave / WN;
  const uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  uint32_t tm, tn;
  tile_of(a, id, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * CH;
  const Operands& op = a.op;

  // Of a pair, channels 8 c .. 8 c + 7 are the tile's rows 16 c .. 16 c + 7, and those of
  // the second matrix the next eight: a lane has both of a channel in its registers.
  RowLoader<BN, NW, EPI == kGate> lw;
  RowLoader<BM, NW> lx;
  if (EPI == kGate && (wave & 1))
    lw.init(a.act.Wu, a.act.ldwu, n0, op.N, op.K, wave, lane);
  else
    lw.init(op.W, op.ldw, n0, op.N, op.K, wave, lane);
  lx.init(op.X, op.ldx, m0, op.M, op.K, wave, lane);
  uint8_t* mine = lds + group * DEPTH * S::kBytes;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)mine;

  for (int i = t; i < BN; i += T) {
    const bool second = EPI == kGate && (i & 8);
    const int64_t n = n0 + (EPI == kGate ? 8 * (i >> 4) + (i & 7) : i);
    const bool in = n < op.N;
    swl[i] = in ? (second ? a.act.swu : op.sw)[n] : 0.0f;
    if constexpr (kBiased) {
      const float* b = EPI == kLinear ? a.lin.bias : second ? a.act.biasu : a.act.bias;
      bias[i] = in && b ? b[n] : 0.0f;
    }
  }

  v16i acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  constexpr int kLw = decltype(lw)::kIssues, kLoads = kLw + RowLoader<BM, NW>::kIssues;
  // load j of this wave's kLoads for a step
  auto load = [&](int j, uint32_t take, int k0, uint32_t back, uint32_t to) {
    if (j < kLw)
      lw.issue(j, take, k0, back, to + S::kW, wave);
    else
      lx.issue(j - kLw, take, k0, back, to + S::kX, wave);
  };

  // Fragments of a quarter step (32 bytes of K): two sets, one read while the
  // matrix cores work on the other.
  v4i wf[2][TN], xf[2][TM];
  constexpr int kReads = TN + TM, kProducts = TN * TM;
  auto read = [&](const uint8_t* stage, int q, int r) {
    if (r < TN)
      wf[q & 1][r] = frag(stage + S::kW, (wn * TN + r) * 32 + (lane & 31), 2 * q + (lane >> 5));
    else
      xf[q & 1][r - TN] =
          frag(stage + S::kX, (wm * TM + r - TN) * 32 + (lane & 31), 2 * q + (lane >> 5));
  };
  // The products of quarter q, with the reads of the next quarter over the first
  // half of them and, in quarter 3, the loads of a later step over all: each is
  // issued while an MFMA runs.  A burst of either would leave the matrix cores
  // idle behind it.  Everything in one loop body, with the branches around the
  // loads inside their asm: a second copy of the products makes the compiler move
  // all accumulators between the two.
  constexpr int kPerProduct = (2 * kReads + kProducts - 1) / kProducts;
  auto quarter = [&](int q, const uint8_t* from, uint32_t take, int k0, uint32_t back,
                     uint32_t to) {
#pragma unroll
    for (int p = 0; p < kProducts; ++p) {
      acc[p / TM][p % TM] =
          gk::mfma_i8(wf[q & 1][p / TM], xf[q & 1][p % TM], acc[p / TM][p % TM]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = p * kPerProduct; r < (p + 1) * kPerProduct && r < kReads; ++r)
        read(from, (q + 1) & 3, r);
      if (q == 3) {
#pragma unroll
        for (int j = p * kLoads / kProducts; j < (p + 1) * kLoads / kProducts; ++j)
          load(j, take, k0, back, to);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // local step s of the group is step s GROUPS + group of K; every group goes
  // through `steps` of them, some through one past the end, which adds zero
  const int all = (op.K + kStep - 1) / kStep;
  const int steps = (all + GROUPS - 1) / GROUPS, own = (all - group + GROUPS - 1) / GROUPS;
  auto column = [&](int s) { return (s * GROUPS + group) * kStep; };
  // the last local step's columns from K on are cleared, by its own group
  auto clear_last = [&](uint8_t* stage) {
    if (op.K % kStep || all % GROUPS) {
      clear_tail<BM, 64 * NW>(stage + S::kX, column(steps - 1), op.K, t % (64 * NW));
      gk::lds_barrier();
    }
  };

#pragma unroll
  for (int s = 0; s < DEPTH; ++s) {
    const uint32_t back = lw.over(column(s));
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      load(j, s < own, column(s), back, lds0 + s * S::kBytes);
  }
  wait_vm_if<(DEPTH - 1) * kLoads>(own >= DEPTH);
  gk::lds_barrier();
  if (steps == 1) clear_last(mine);
#pragma unroll
  for (int r = 0; r < kReads; ++r) read(mine, 0, r);

  // Past the barrier in step s the next step is in LDS (the loads of DEPTH - 2
  // later ones may be under way) and every wave has read all of this one, so that
  // its buffer takes the step DEPTH further on.  The last step reads a buffer that
  // it does not use.
  int buf = 0;
  for (int s = 0; s < steps; ++s) {
    const int nbuf = buf == DEPTH - 1 ? 0 : buf + 1;
    const uint8_t* cur = mine + buf * S::kBytes;
    uint8_t* next = mine + nbuf * S::kBytes;
#pragma unroll
    for (int q = 0; q < 3; ++q) quarter(q, cur, 0, 0, 0, 0);
    wait_vm_if<(DEPTH - 2) * kLoads>(s + DEPTH - 1 < own);
    gk::lds_barrier();
    if (s + 2 == steps) clear_last(next);
    const int k0 = column(s + DEPTH);
    quarter(3, next, s + DEPTH < own, k0, lw.over(k0), lds0 + buf * S::kBytes);
    buf = nbuf;
  }
  gk::lds_barrier();  // no wave still reads what follows writes

  if constexpr (GROUPS > 1) {
    constexpr int kAt = BM * BN * 2;  // behind the results' image
    static_assert(kAt + (GROUPS - 1) * BM * BN * 4 <= GROUPS * DEPTH * S::kBytes, "the sums fit");
    v4i* sums = reinterpret_cast<v4i*>(lds + kAt);
    auto at = [&](int g, int i, int j, int r) {
      return ((((g - 1) * NW + wave) * TN + i) * TM + j) * 256 + r * 64 + lane;
    };
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sums[at(group, i, j, r)] = (v4i){acc[i][j][4 * r], acc[i][j][4 * r + 1],
                                             acc[i][j][4 * r + 2], acc[i][j][4 * r + 3]};
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < GROUPS; ++g)
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int j = 0; j < TM; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const v4i o = sums[at(g, i, j, r)];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][j][4 * r + e] += o[e];
            }
    }
  }

  // Lane l holds token 32 (wm TM + j) + (l & 31) and, in registers 4 g .. 4 g + 3
  // of tile i, channels 32 (wn TN + i) + 8 g + 4 (l >> 5) + 0..3.
  const int h = lane >> 5, nw = wn * TN * 32 + 4 * h;
  const bool edge = n0 + CH > op.N;  // some of the tile's channels do not exist
  if constexpr (EPI == kAct || EPI == kGate) {
    static_assert(BM * CH * 2 <= GROUPS * DEPTH * S::kBytes, "the results fit the steps' buffers");
    finish_act<BN, BM, WN, WM, T, EPI>(a, acc, swl, bias, lds, m0, n0, wn, wm, lane, group, t);
    return;
  }
  // 16-bit results go through LDS, so that rows are written in whole lines.  Written
  // from the registers, four values of a token at a time and 32 tokens an
  // instruction, the factor of M = 1024 by 50688 rows took 200 us instead of 160.
  constexpr int kChunks = Image<BN>::kChunks, kMix = Image<BN>::kMix;
  static_assert(BM * BN * 2 <= GROUPS * DEPTH * S::kBytes, "the results fit the steps' buffers");
  bool staged = false;
  if constexpr (EPI == kLinear) staged = a.lin.type != GEMMQ_F32;
  if constexpr (EPI == kFactor) staged = a.fac.planes == 1;
  auto put = [&](int ml, int nl, uint32_t lo, uint32_t hi) {
    *reinterpret_cast<uint2*>(lds + (ml * kChunks + ((nl >> 3) ^ (ml & kMix))) * 16 +
                              8 * h) = make_uint2(lo, hi);
  };
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    if (group > 0) break;
    const int ml = (wm * TM + j) * 32 + (lane & 31);
    const int64_t m = m0 + ml;
    const bool inside = m < op.M;
    const float sx = inside ? op.sx[m] : 0.0f;
    if constexpr (EPI == kLinear) {
      if (!inside) continue;
      const bool wide = a.lin.wide && !edge;
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int nl = nw + 32 * i + 8 * g;
          const float4 sw = *reinterpret_cast<const float4*>(swl + nl);
          const float4 b = *reinterpret_cast<const float4*>(bias + nl);
          const v16i& c = acc[i][j];
          const float v0 = fmaf((float)c[4 * g] * sx, sw.x, b.x);
          const float v1 = fmaf((float)c[4 * g + 1] * sx, sw.y, b.y);
          const float v2 = fmaf((float)c[4 * g + 2] * sx, sw.z, b.z);
          const float v3 = fmaf((float)c[4 * g + 3] * sx, sw.w, b.w);
          const int64_t n = n0 + nl;
          if (staged) {
            if (a.lin.type == GEMMQ_BF16)
              put(ml, nl, bf16_bits(v0) | bf16_bits(v1) << 16, bf16_bits(v2) | bf16_bits(v3) << 16);
            else
              put(ml, nl, f16_bits(v0) | f16_bits(v1) << 16, f16_bits(v2) | f16_bits(v3) << 16);
          } else {
            store4_as(a.lin.Y, m * a.lin.ldy + n, a.lin.type, wide,
                      edge ? (int)min((int64_t)4, op.N - n) : 4, v0, v1, v2, v3);
          }
        }
    } else {
      // base-2 logits, exp(z) = 2^(z log2 e): v = sw I, z2 = s2 v with s2 = sx log2 e.
      // A negative scale is moved to v, so that the largest v has the largest logit.
      float s2 = sx * kLog2e;
      const float sign = s2 < 0.0f ? -1.0f : 1.0f;
      s2 *= sign;
      // the factor's target among the lane's channels, and its sum, here where the sums
      // are still at hand.  The asm keeps the comparisons one after another: all at
      // once their masks do not fit the scalar registers.
      int tg = -1, dot = 0;
      if constexpr (EPI == kFactor) {
        if (inside) {
          // (one past the operands' rows is a later piece's, or no token's)
          const int64_t in = a.fac.target[m] - a.fac.n0, at = in - n0 - wn * TN * 32;
          if (at >= 0 && at < TN * 32 && in < op.N) tg = (int)at;
        }
        tg = (tg >> 2 & 1) == h ? tg - 4 * h : -1;
        if (tg >= 0) {
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              dot = tg == 32 * i + 8 * (r >> 2) + (r & 3) ? acc[i][j][r] : dot;
              if ((r & 3) == 3) asm volatile("" : "+v"(tg), "+v"(dot));
            }
        }
      }
      float v[TN][16];
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float4 sw = *reinterpret_cast<const float4*>(swl + nw + 32 * i + 8 * g);
          v[i][4 * g] = (float)acc[i][j][4 * g] * sw.x;
          v[i][4 * g + 1] = (float)acc[i][j][4 * g + 1] * sw.y;
          v[i][4 * g + 2] = (float)acc[i][j][4 * g + 2] * sw.z;
          v[i][4 * g + 3] = (float)acc[i][j][4 * g + 3] * sw.w;
        }
      if (__any(sign < 0.0f)) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) v[i][r] *= sign;
      }
      if constexpr (EPI == kLoss) {
        if (edge) {
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (n0 + nw + 32 * i + 8 * (r >> 2) + (r & 3) >= op.N) v[i][r] = -__builtin_inff();
        }
        // A NaN is dropped by the maximum and kept by the sum.  A wave whose
        // columns all lie past N takes 0 as its maximum, and has the sum 0.  The sum is
        // of exp2((v - top) s2), the largest term exactly 1 (with v s2 - top s2 in one
        // step, top s2 rounded, the sum is off by |z| 2^-24).
        float top = v[0][0];
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r) top = fmaxf(top, v[i][r]);
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float v0 = top == -__builtin_inff() ? 0.0f : top;
        float sum = 0.0f;
        if (edge) {
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              if (n0 + nw + 32 * i + 8 * (r >> 2) + (r & 3) < op.N)
                sum += __builtin_amdgcn_exp2f((v[i][r] - v0) * s2);
        } else {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r)
              part[r & 3] += __builtin_amdgcn_exp2f((v[i][r] - v0) * s2);
          sum = (part[0] + part[1]) + (part[2] + part[3]);
        }
        sum += __shfl_xor(sum, 32, 64);
        if (h == 0) red[wn * BM + ml] = make_float2(top, sum);
      } else {
        if (!inside) continue;
        // the difference first, in units of e and rounded once, then the change to base
        // 2: lse log2 e rounded would put all of a row off by |lse| 2^-24
        const float lse = a.fac.lse[m], sx1 = sx * sign;
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            v[i][r] = __builtin_amdgcn_exp2f(fmaf(v[i][r], sx1, -lse) * kLog2e);
        if (tg >= 0) {
          const float sw = swl[nw + tg], less = target_factor(dot, sw, sx, lse);
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              v[i][r] = tg == 32 * i + 8 * (r >> 2) + (r & 3) ? less : v[i][r];
              if ((r & 3) == 3) asm volatile("" : "+v"(tg));
            }
          if (a.fac.rest) a.fac.rest[m] = bf16_rest(less * sw);
        }
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int nl = nw + 32 * i + 8 * g;
            const float4 sw = *reinterpret_cast<const float4*>(swl + nl);
            float(&f)[16] = v[i];
            f[4 * g] *= sw.x, f[4 * g + 1] *= sw.y, f[4 * g + 2] *= sw.z, f[4 * g + 3] *= sw.w;
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n0 + nl + e >= op.N) f[4 * g + e] = 0.0f;
            }
            if (staged)
              put(ml, nl, bf16_bits(f[4 * g]) | bf16_bits(f[4 * g + 1]) << 16,
                  bf16_bits(f[4 * g + 2]) | bf16_bits(f[4 * g + 3]) << 16);
          }
        // More planes, from the registers: lanes l and l + 32 hold a token's channels
        // 0-3 and 4-7 of eight; of two such groups the lower lane takes the first
        // whole and the upper one the second, 16 bytes each and 32 next to each other
        // (three planes of 1000 x 32000: 158 -> 120 us; through LDS as above, a plane
        // at a time, 155).  With one 32-channel tile a wave the values as they lie are
        // faster (37 x 32003: 11 us, exchanged 13).
        if (!staged) {
          const int64_t plane = (int64_t)op.M * a.fac.pitch;
#pragma unroll
          for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
              float(&f)[16] = v[i];
              if constexpr (TN == 1) {
#pragma unroll
                for (int u = g; u < g + 2; ++u) {
                  float w[4] = {f[4 * u], f[4 * u + 1], f[4 * u + 2], f[4 * u + 3]};
                  const int64_t n = n0 + nw + 8 * u;
                  if (n < a.fac.pitch)  // a multiple of 64
                    store_planes(a.fac.P + m * a.fac.pitch + n, plane, a.fac.planes, w);
                }
              } else {
                const int64_t n = n0 + wn * TN * 32 + 32 * i + 8 * (g + h);
                uint16_t* to = a.fac.P + m * a.fac.pitch + n;
                for (int p = 0; p < a.fac.planes; ++p) {
                  uint32_t b[8];
#pragma unroll
                  for (int e = 0; e < 8; ++e)
                    b[e] = bf16_part(f[4 * g + e], p + 1 == a.fac.planes);
                  const v2u lo = swap_halves(b[0] | b[1] << 16, b[4] | b[5] << 16);
                  const v2u hi = swap_halves(b[2] | b[3] << 16, b[6] | b[7] << 16);
                  if (n < a.fac.pitch)
                    *reinterpret_cast<uint4*>(to + p * plane) =
                        make_uint4(lo[0], hi[0], lo[1], hi[1]);
                }
              }
            }
        }
      }
    }
  }
  if constexpr (EPI != kLoss) {
    if (staged) {
      uint16_t* out;
      int64_t pitch, width;  // the width of a row that is written
      if constexpr (EPI == kLinear) {
        out = static_cast<uint16_t*>(a.lin.Y), pitch = a.lin.ldy, width = op.N;
      } else {
        out = a.fac.P, pitch = a.fac.pitch, width = a.fac.pitch;
      }
      __syncthreads();
      bool lines = true;
      if constexpr (EPI == kLinear) lines = a.lin.lines;
      if (lines) {
        for (int i = t; i < BM * kChunks; i += T) {
          const int ml = i / kChunks, c = i % kChunks;
          const int64_t n = n0 + 8 * c;
          if (m0 + ml >= op.M || n >= width) continue;
          const v4i v = *reinterpret_cast<const v4i*>(
              lds + (ml * kChunks + (c ^ (ml & kMix))) * 16);
          uint16_t* to = out + (m0 + ml) * pitch + n;
          if (n + 8 <= width) {
            *reinterpret_cast<v4i*>(to) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (n + e < width) to[e] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
          }
        }
      } else {
        // rows off 16 bytes: neighbouring lanes still write neighbouring values
        for (int i = t; i < BM * BN; i += T) {
          const int ml = i / BN, nl = i % BN;
          if (m0 + ml >= op.M || n0 + nl >= width) continue;
          out[(m0 + ml) * pitch + n0 + nl] = *reinterpret_cast<const uint16_t*>(
              lds + (ml * kChunks + ((nl >> 3) ^ (ml & kMix))) * 16 + 2 * (nl & 7));
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
      for (int w = 1; w < WN; ++w) top = fmaxf(top, red[w * BM + ml].x);
      float sum = 0.0f;
      const float s2 = fabsf(op.sx[m0 + ml]) * kLog2e;
#pragma unroll
      for (int w = 0; w < WN; ++w) sum += join_term(red[w * BM + ml], top, s2);
      a.loss.part[(m0 + ml) * a.loss.ntiles + n0 / BN] = make_float2(top, sum);
    }
  }
}

constexpr int kCUs = 256;

// A tile, its groups of waves, the waves of a group, and the time of a K step (us) on
// a compute unit that works on one, two or three such workgroups at a time, 0 where
// its LDS holds fewer.  A step waits for its loads: the times are near 64 bytes a
// nanosecond where much is in flight, and never below the 0.42 us of a round trip.
struct Tile {
  int bn, bm, groups, waves;
  float step[3];
};
constexpr Tile kTiles[] = {
    {256, 256, 1, 8, {1.55f, 0, 0}},       {128, 256, 1, 8, {1.02f, 0, 0}},
    {192, 128, 1, 8, {0.86f, 0, 0}},       {128, 128, 1, 8, {0.70f, 1.05f, 0}},
    {128, 128, 1, 8, {0.66f, 0, 0}},       {128, 64, 1, 4, {0.50f, 0.70f, 1.0f}},
    {64, 64, 1, 4, {0.43f, 0.50f, 0.75f}}, {64, 64, 2, 4, {0.74f, 0.88f, 0}},
    {64, 32, 4, 2, {0.85f, 0, 0}},         {64, 32, 1, 2, {0.42f, 0.45f, 0.6f}},
    {128, 32, 1, 4, {}}};
constexpr int kMaxThreads = 512;
constexpr int kTileCount = 10;  // of those that pick_tile compares
constexpr int kWideTile = 10;

inline int64_t tiles(const Tile& c, int M, int N) { return ceil_div(M, c.bm) * ceil_div(N, c.bn); }

// The tile with the least estimated time: rounds of the chip, each of the K steps,
// 2 us around them, and 0.08 ns for an output, more where fewer than eight waves (two
// a SIMD) write them: the groups' sums are one group's to finish.  Measured (us,
// random int8 data; tiles in the order of kTiles, the one taken in brackets):
//   M 4096 N 4096 K 4096   [63] 74   80    72    85    87   106   115
//   M 2048 N 4096 K 12288  127 [102] 147   104   136   155  183   177
//   M 512 N 12288 K 4096   51   37  [32]   34    45    36   45    46
//   M 1504 N 5008 K 2560   36  [27]  36    26    31    36   37    41
//   M 1024 N 4096 K 4096   49   34   28    28   [25]   26   33    31
//   M 64 N 151936 K 2048   -    -    82    76    78   [69]  67    72    120   81
//   M 512 N 4096 K 4096    45   30   26    24    22    22   18.5 [16.6]
//   M 64 N 32000 K 4096    -    -    26    28    25    31   22.3 [22.2] 33    30
//   M 128 N 4096 K 4096                                17   14    11   [9]    15
// Up to 32 tokens of a vocabulary W's stream decides, and 128 channels a workgroup are
// ahead of 64 once there are more than three such workgroups a CU, 98304 channels (the
// loss at M = 8 over K = 2048, 128 / 64 channels: N = 66000 31.3 / 28.5 us, 80000 33.0 /
// 32.0, 98304 36.2 / 36.9, 115000 41.1 / 44.2, 151936 56.6 / 58.5, 200000 79.9 / 88.1).
inline int pick_tile(int M, int N, int K) {
  if (M <= 32 && N > 98304) return kWideTile;
  const int64_t steps = ceil_div(K, kStep);
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < kTileCount; ++i) {
    const Tile& c = kTiles[i];
    const int64_t n = tiles(c, M, N);
    int r = 1;
    while (r < 3 && c.step[r] > 0.0f && n > kCUs * r) ++r;
    const double rounds = (double)ceil_div(n, kCUs * r);
    const int writers = r * c.waves < 8 ? r * c.waves : 8;
    const double t = rounds * ((double)ceil_div(steps, c.groups) * c.step[r - 1] + 2.0 +
                               0.64e-3 / writers * r * c.bn * c.bm);
    if (i == 0 || t < least) {
      best = i;
      least = t;
    }
  }
  return best;
}

// Up to 16 tokens: the stream into registers, whose waves share a workgroup's K,
// where the tiles would be too few to fill the chip (us, stream / tiles: M = 8,
// 4096 x 4096 5.9 / 8; M = 16, 12288 x 4096 13 / 16).  `linear` at M <= 4 also
// beyond (151936 x 2048 at M = 1 53 / 58, M = 4 57 / 59); the loss would have
// more partial sums to join there.
inline bool skinny(int M, int N, bool linear) {
  return M <= kSkinnyMaxM && (N <= 16384 || (M <= 4 && linear));
}

template <int EPI>
int launch_tiles(TileArgs& a, hipStream_t st) {
  const int rows = EPI == kGate ? 2 * a.op.N : a.op.N;  // of W, or of both matrices
  const int pick = pick_tile(a.op.M, rows, a.op.K);
  const Tile& c = kTiles[pick];
  const int64_t n = tiles(c, a.op.M, rows);
  if (!grid_fits(n, kMaxThreads)) return -1;
  a.mtiles = (uint32_t)ceil_div(a.op.M, c.bm);
  a.ntiles = (uint32_t)ceil_div(rows, c.bn);
  a.group = 1024 / c.bm;
  const dim3 grid((uint32_t)n);
  switch (pick) {
    case 0: tile_kernel<256, 256, 2, 4, 2, 1, EPI><<<grid, 512, 0, st>>>(a); break;
    case 1: tile_kernel<128, 256, 2, 4, 3, 1, EPI><<<grid, 512, 0, st>>>(a); break;
    case 2: tile_kernel<192, 128, 2, 4, 3, 1, EPI><<<grid, 512, 0, st>>>(a); break;
    case 3: tile_kernel<128, 128, 2, 4, 2, 1, EPI><<<grid, 512, 0, st>>>(a); break;
    case 4: tile_kernel<128, 128, 2, 4, 4, 1, EPI><<<grid, 512, 0, st>>>(a); break;
    case 5: tile_kernel<128, 64, 2, 2, 2, 1, EPI><<<grid, 256, 0, st>>>(a); break;
    case 6: tile_kernel<64, 64, 2, 2, 3, 1, EPI><<<grid, 256, 0, st>>>(a); break;
    case 7: tile_kernel<64, 64, 2, 2, 2, 2, EPI><<<grid, 512, 0, st>>>(a); break;
    case 8: tile_kernel<64, 32, 2, 1, 3, 4, EPI><<<grid, 512, 0, st>>>(a); break;
    case 9: tile_kernel<64, 32, 2, 1, 4, 1, EPI><<<grid, 128, 0, st>>>(a); break;
    default: tile_kernel<128, 32, 4, 1, 3, 1, EPI><<<grid, 256, 0, st>>>(a); break;
  }
  return 0;
}

}  // namespace
}  // namespace i8
}  // namespace gemmq
