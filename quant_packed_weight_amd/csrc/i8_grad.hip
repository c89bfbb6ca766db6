// i8_grad.hip -- the product that both gradients need, acc[m, k] = sum_n
// A[m, n] W[n, k]: int8 weights, exact in bf16, against a factor A given as one
// to three bf16 matrices whose sum it is; and the kernels before and after it.
//
// W is read as it lies, rows of N along the reduction: the transposing LDS read
// hands each lane the eight consecutive n of its own k, which are converted to
// bf16 in registers (int8 is exact there), so LDS and the loads hold one byte per
// weight.  W^T is the MFMA's row operand: a lane ends with one token and four
// consecutive k per register quad.
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

constexpr int kRed = 64;  // n per step: kRed rows of W's tile, 128 bytes of A's rows

__device__ __forceinline__ v16f mfma_bf16(v8bf a, v8bf b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// eight int8 to bf16, exactly
__device__ __forceinline__ v8bf widen(v2i w) {
  v8bf r;
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = (__bf16)(float)(int8_t)(w[e >> 2] >> (8 * (e & 3)));
  return r;
}

template <int BK, int BM>
struct GradStage {
  static constexpr int kW = 0, kA = kRed * BK, kBytes = kRed * BK + BM * 2 * kRed;
};

// W's LDS image: rows of BK bytes, chunk c of row n in slot c ^ 2 (n & 7): the
// eight rows by two chunks that 32 lanes of a transposing read take lie in 16
// different columns of 256 bytes.  (BK >= 256; rows of 128 bytes lie two to that
// span, and take c ^ 2 ((n >> 1) & 3) instead.)
template <int BK>
__device__ __forceinline__ int wslot(int n, int chunk) {
  return BK >= 256 ? chunk ^ ((n & 7) << 1) : chunk ^ (((n >> 1) & 3) << 1);
}
// A's image: as the int8 product's operands (i8_gemm.hip)
__device__ __forceinline__ int aslot(int m, int chunk) { return chunk ^ ((m >> 1) & 7); }

template <int BK, int BM, int WK, int WM, int DEPTH>
__global__ __launch_bounds__(64 * WK * WM, 2) void grad_kernel(GradArgs a, uint32_t ktiles,
                                                               uint32_t mtiles) {
  constexpr int NW = WK * WM;
  constexpr int TK = BK / WK / 32, TM = BM / WM / 32;
  using S = GradStage<BK, BM>;
  constexpr int kRowsPer = 1024 / BK;  // rows of W per load
  constexpr int kLw = kRed / kRowsPer / NW, kLa = BM / 8 / NW, kLoads = kLw + kLa;
  static_assert(kLw * kRowsPer * NW == kRed && kLa * 8 * NW == BM && NW % 2 == 0,
                "every wave issues the same loads");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[DEPTH * S::kBytes];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wk = wave % WK, wm = wave / WK;
  uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(id % mtiles) * BM;
  id /= mtiles;
  const int k0 = (int)(id % ktiles) * BK, split = (int)(id / ktiles);

  // this split's share of the steps of kRed rows; every plane goes over it
  const int steps = (a.N + kRed - 1) / kRed;
  const int per = steps / a.splits, more = steps % a.splits;
  const int first = split * per + min(split, more), count = per + (split < more ? 1 : 0);
  const int its = count * a.planes;

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int mvalid = (int)min((int64_t)BM, a.M - m0);
  const uint32_t arow = (uint32_t)(2 * a.pitch);
  int wrow[kLw];
  uint32_t wcol[kLw], aoff[kLa];
#pragma unroll
  for (int j = 0; j < kLw; ++j) {
    const int r = kRowsPer * (wave + NW * j) + lane / (BK / 16);
    wrow[j] = r;
    // chunks past column K repeat the last one: their columns are dropped
    wcol[j] = (uint32_t)min(k0 + 16 * wslot<BK>(r, lane % (BK / 16)), (a.K - 1) / 16 * 16);
  }
#pragma unroll
  for (int j = 0; j < kLa; ++j) {
    const int r = 8 * (wave + NW * j) + (lane >> 3);
    // rows past the last token repeat it: their results are dropped
    aoff[j] = (uint32_t)min(r, mvalid - 1) * arow + 16 * aslot(r, lane & 7);
  }
  // iteration `it` reads step first + it / planes of plane it % planes; `ahead`
  // is the one that is loaded next
  int astep = first, aplane = 0;
  auto load = [&](int j, uint32_t take, uint32_t to) {
    const int64_t n = (int64_t)min(astep, steps - 1) * kRed;
    if (j < kLw) {
      // rows of W past the last one repeat it: the factor is zero there
      const int nvalid = (int)min((int64_t)kRed, a.N - n);
      const rsrc_t rs = gk::make_rsrc(a.W + n * a.ldw, (uint32_t)(nvalid * a.ldw));
      gk::dma16_if(take, rs, (uint32_t)(min(wrow[j], nvalid - 1) * (int)a.ldw) + wcol[j], 0,
                   to + S::kW + 1024 * (wave + NW * j));
    } else {
      const rsrc_t rs = gk::make_rsrc(a.P + ((int64_t)aplane * a.M + m0) * a.pitch,
                                      (uint32_t)mvalid * arow);
      gk::dma16_if(take, rs, aoff[j - kLw], (uint32_t)(2 * n),
                   to + S::kA + 1024 * (wave + NW * (j - kLw)));
    }
  };
  auto advance = [&] {
    if (++aplane == a.planes) {
      aplane = 0;
      ++astep;
    }
  };

  v16f acc[TK][TM];
#pragma unroll
  for (int i = 0; i < TK; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Two sets of fragments of a quarter step (16 n), as in the int8 product.  The
  // transposing read: of each 16 lanes, lanes 2 r and 2 r + 1 give the addresses
  // of the two halves of 16 k of row r, and lane i takes k i of the eight rows.
  v2i wraw[2][TK];
  v8bf af[2][TM];
  constexpr int kReads = TK + TM, kProducts = TK * TM;
  constexpr int kPerProduct = (2 * kReads + kProducts - 1) / kProducts;
  const int h = lane >> 5;
  auto read = [&](int stage, int q, int r) {
    if (r < TK) {
      const int n = 16 * q + 8 * h + ((lane & 15) >> 1);
      const int c = 2 * (wk * TK + r) + ((lane >> 4) & 1);
      const uint8_t* p = lds + stage * S::kBytes + S::kW + n * BK + 16 * wslot<BK>(n, c) +
                         8 * (lane & 1);
      wraw[q & 1][r] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) v2i*)p);
    } else {
      const int m = (wm * TM + r - TK) * 32 + (lane & 31);
      af[q & 1][r - TK] = *reinterpret_cast<const v8bf*>(
          lds + stage * S::kBytes + S::kA + m * 2 * kRed + 16 * aslot(m, 2 * q + h));
    }
  };
  auto quarter = [&](int q, int from, uint32_t take, uint32_t to) {
#pragma unroll
    for (int i = 0; i < TK; ++i) {
      const v8bf w = widen(wraw[q & 1][i]);
#pragma unroll
      for (int j = 0; j < TM; ++j) {
        const int p = i * TM + j;
        acc[i][j] = mfma_bf16(w, af[q & 1][j], acc[i][j]);
        if (j == TM - 1) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = p * kPerProduct; r < (p + 1) * kPerProduct && r < kReads; ++r)
          read(from, (q + 1) & 3, r);
        if (q == 3) {
#pragma unroll
          for (int l = p * kLoads / kProducts; l < (p + 1) * kLoads / kProducts; ++l)
            load(l, take, to);
        }
      }
    }
  };

#pragma unroll
  for (int s = 0; s < DEPTH; ++s) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(j, s < its, lds0 + s * S::kBytes);
    advance();
  }
  if (its > 0) {
    wait_vm_if<(DEPTH - 1) * kLoads>(its >= DEPTH);
    gk::lds_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, 0, r);
  }
  int buf = 0;
  for (int it = 0; it < its; ++it) {
    const int nbuf = buf == DEPTH - 1 ? 0 : buf + 1;
#pragma unroll
    for (int q = 0; q < 3; ++q) quarter(q, buf, 0, 0);
    wait_vm_if<(DEPTH - 2) * kLoads>(it + DEPTH - 1 < its);
    gk::lds_barrier();
    quarter(3, nbuf, it + DEPTH < its, lds0 + buf * S::kBytes);
    advance();
    buf = nbuf;
  }

#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + (wm * TM + j) * 32 + (lane & 31);
    if (m >= a.M) continue;
    float* out = a.acc + ((int64_t)split * a.M + m) * a.kp;
#pragma unroll
    for (int i = 0; i < TK; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int k = k0 + (wk * TK + i) * 32 + 8 * g + 4 * h;
        if (k >= a.kp) continue;
        float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                               acc[i][j][4 * g + 3]);
        float4* p = reinterpret_cast<float4*>(out + k);
        if (a.add) {
          const float4 o = *p;
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        *p = v;
      }
  }
}

// A[m, n] = dY[m, n] * sw[n] as `planes` bf16 matrices, zero from column N to
// the pitch.  One thread per four columns.
__global__ __launch_bounds__(256) void planes_kernel(int type, const void* dY, int64_t lddy,
                                                     const float* sw, uint16_t* P, int64_t pitch,
                                                     int planes, int M, int N) {
  const int64_t q = pitch / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / q;
  if (m >= M) return;
  const int64_t n = 4 * (i % q);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = n + e < N ? load_as_f32(dY, m * lddy + n + e, type) * sw[n + e] : 0.0f;
  for (int p = 0; p < planes; ++p) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = bf16_part(v[e], p + 1 == planes);
    *reinterpret_cast<uint2*>(P + ((int64_t)p * M + m) * pitch + n) =
        make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  }
}

__global__ __launch_bounds__(256) void finish_kernel(const float* acc, int64_t kp, int splits,
                                                     const float* g, const int64_t* target,
                                                     int64_t nvocab, int type, void* dX,
                                                     int64_t lddx, int M, int K) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / K;
  if (m >= M) return;
  const int64_t k = i % K;
  float v = 0.0f;
  for (int s = 0; s < splits; ++s) v += acc[((int64_t)s * M + m) * kp + k];
  if (g) v *= g[m];
  if (target) {
    const int64_t tg = target[m];
    v = tg < 0 ? 0.0f : tg >= nvocab ? __builtin_nanf("") : v;
  }
  store_as(dX, m * lddx + k, type, v);
}

constexpr int64_t kMaxGrid = 0x7fffffff;

struct Tile {
  int bk, bm;
};
Tile pick_tile(int M) { return M <= 32 ? Tile{128, 32} : M <= 128 ? Tile{128, 128} : Tile{256, 256}; }

int64_t tiles(int M, int K) {
  const Tile c = pick_tile(M);
  return ceil_div(M, c.bm) * ceil_div(K, c.bk);
}

}  // namespace

int grad_splits(int M, int N, int K, int) {
  const int64_t steps = ceil_div(N, kRed);
  int64_t s = ceil_div(256, tiles(M, K));
  if (s > steps / 4) s = steps / 4;
  return s < 1 ? 1 : (int)s;
}

bool grad_fits(int M, int K, int splits) {
  return tiles(M, K) * splits <= kMaxGrid && ceil_div((int64_t)M * K, 256) <= kMaxGrid;
}

int launch_grad(const GradArgs& a, hipStream_t st) {
  const Tile c = pick_tile(a.M);
  const int64_t mt = ceil_div(a.M, c.bm), kt = ceil_div(a.K, c.bk), n = mt * kt * a.splits;
  if (n > kMaxGrid) return -1;
  if (c.bm == 32)
    grad_kernel<128, 32, 4, 1, 3><<<(uint32_t)n, 256, 0, st>>>(a, (uint32_t)kt, (uint32_t)mt);
  else if (c.bm == 128)
    grad_kernel<128, 128, 2, 2, 3><<<(uint32_t)n, 256, 0, st>>>(a, (uint32_t)kt, (uint32_t)mt);
  else
    grad_kernel<256, 256, 4, 2, 3><<<(uint32_t)n, 512, 0, st>>>(a, (uint32_t)kt, (uint32_t)mt);
  return 0;
}

int launch_planes(int type, const void* dY, int64_t lddy, const float* sw, uint16_t* P,
                  int64_t pitch, int planes, int M, int N, hipStream_t st) {
  const int64_t n = ceil_div(M * (pitch / 4), 256);
  if (n > kMaxGrid) return -1;
  planes_kernel<<<(uint32_t)n, 256, 0, st>>>(type, dY, lddy, sw, P, pitch, planes, M, N);
  return 0;
}

int launch_finish(const float* acc, int64_t kp, int splits, const float* g, const int64_t* target,
                  int64_t nvocab, int type, void* dX, int64_t lddx, int M, int K,
                  hipStream_t st) {
  finish_kernel<<<(uint32_t)ceil_div((int64_t)M * K, 256), 256, 0, st>>>(
      acc, kp, splits, g, target, nvocab, type, dX, lddx, M, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
