// i8_grad.hip -- the product that both gradients need, acc[m, k] = sum_n
// A[m, n] W[n, k]: int8 weights, exact in bf16, against a factor A given as one
// to three bf16 matrices whose sum it is, or as the caller's own bf16 rows, which sw
// scales here: the weights, rounded to bf16, or for few rows A itself, in two numbers;
// and the kernels before and after it.
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

// two int8 of w (bytes 2 i and 2 i + 1) to bf16, exactly, or times s0 and s1, rounded.
// The conversion takes the byte out of its word itself (written as source, the odd
// bytes cost a shift each).
template <int i, bool SCALED>
__device__ __forceinline__ uint32_t widen2(int w, float s0, float s1) {
  float lo, hi;
  if constexpr (i == 0) {
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
        : "=v"(lo) : "v"(w));
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
        : "=v"(hi) : "v"(w));
  } else {
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
        : "=v"(lo) : "v"(w));
    asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
        : "=v"(hi) : "v"(w));
  }
  if constexpr (SCALED) {
    lo *= s0;
    hi *= s1;
  }
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf r = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, r);
}
// part e (0..3) of a fragment of eight, their scales s
template <bool SCALED>
__device__ __forceinline__ uint32_t widen_part(v2i w, const float (&s)[8], int e) {
  switch (e) {
    case 0: return widen2<0, SCALED>(w[0], s[0], s[1]);
    case 1: return widen2<1, SCALED>(w[0], s[2], s[3]);
    case 2: return widen2<0, SCALED>(w[1], s[4], s[5]);
    default: return widen2<1, SCALED>(w[1], s[6], s[7]);
  }
}

// How the factor A comes: kPlanes, PLANES matrices in the workspace.  The others are the
// caller's own matrix of bf16, N a multiple of 8: kScaledW, W's rows are scaled by sw as
// they are converted, and rounded once; kScaledA, A is, up to kSplitRows rows of it, as
// PLANES numbers that take the place of a step's rows once these are in LDS (M = 8, 4096 x
// 4096 11.5 us, N = 12288 20.1; W scaled 10.9 and 18.0, two matrices in memory 14.1 and 21.0).
constexpr int kSplitRows = 8;
enum Form { kPlanes, kScaledW, kScaledA };

template <int BK, int BM, int PLANES>
struct GradStage {
  static constexpr int kW = 0, kA = kRed * BK, kPlane = BM * 2 * kRed;
  static constexpr int kBytes = kA + PLANES * kPlane;
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

// four values of row m of the result, from column k on
__device__ __forceinline__ void put_result(const GradOut& o, int64_t m, int k, int K, float4 v) {
  const int64_t tg = o.target ? o.target[m] : 0;
  if (o.rest && tg >= 0 && tg < o.nvocab) {
    const float r = o.rest[m];
    const int w = *reinterpret_cast<const int*>(o.W + tg * o.ldw + k);  // inside: pitch % 16 == 0
    v = make_float4(fmaf(r, (float)(int8_t)w, v.x), fmaf(r, (float)(int8_t)(w >> 8), v.y),
                    fmaf(r, (float)(int8_t)(w >> 16), v.z), fmaf(r, (float)(w >> 24), v.w));
  }
  if (o.g) {
    const float f = o.g[m];
    v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
  if (o.target) {
    const float nan = __builtin_nanf("");
    if (tg < 0) v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (tg >= o.nvocab) v = make_float4(nan, nan, nan, nan);
  }
  store4_as(o.dX, m * o.lddx + k, o.type, o.wide, K - k, v.x, v.y, v.z, v.w);
}

// Two waves a SIMD, or the one that four waves with more than half of the LDS are.
template <int BK, int BM, int WAVES, int DEPTH, int PLANES>
constexpr int kWavesPerSimd =
    WAVES <= 4 && DEPTH * GradStage<BK, BM, PLANES>::kBytes > 81920 ? 1 : 2;

// All PLANES planes in a step: W's tile is read and converted once for them (M =
// 2048, 4096 x 4096 in f32 152 us, one plane after another 188).
template <int BK, int BM, int WK, int WM, int DEPTH, int PLANES, Form FORM>
__global__ __launch_bounds__(64 * WK * WM, (kWavesPerSimd<BK, BM, WK * WM, DEPTH, PLANES>)) void
grad_kernel(GradArgs a, uint32_t ktiles, uint32_t mtiles) {
  constexpr bool SCALED = FORM != kPlanes;
  constexpr int kIn = SCALED ? 1 : PLANES;  // matrices that are loaded
  constexpr int NW = WK * WM;
  constexpr int TK = BK / WK / 32, TM = BM / WM / 32;
  static_assert(FORM != kScaledW || PLANES == 1, "the caller's matrix is one");
  static_assert(FORM != kScaledA || 64 * NW == kSplitRows * kRed / 2, "two values a thread");
  using S = GradStage<BK, BM, PLANES>;
  constexpr int kRowsPer = 1024 / BK;  // rows of W per load
  constexpr int kLw = kRed / kRowsPer / NW, kLa = BM / 8 / NW;
  constexpr int kLoads = kLw + kIn * kLa + (SCALED ? 1 : 0);
  static_assert(kLw * kRowsPer * NW == kRed && kLa * 8 * NW == BM && NW % 2 == 0,
                "every wave issues the same loads");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[DEPTH * S::kBytes];
  // a step's scales, each wave its own copy of them
  __shared__ __attribute__((aligned(256))) float swl[SCALED ? DEPTH * NW * kRed : 4];

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wk = wave % WK, wm = wave / WK;
  uint32_t id = xcd_order(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(id % mtiles) * BM;
  id /= mtiles;
  const int k0 = (int)(id % ktiles) * BK, split = (int)(id / ktiles);

  // this split's share of the steps of kRed rows
  const int steps = (a.N + kRed - 1) / kRed;
  const int per = steps / a.splits, more = steps % a.splits;
  const int first = split * per + min(split, more), its = per + (split < more ? 1 : 0);

  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  uint32_t swl0 = 0;
  if constexpr (SCALED)
    swl0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)swl;
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
  // (NW is even: the slot is the same in all of a wave's loads)
  const int achunk = 16 * aslot(8 * (wave & 1) + (lane >> 3), lane & 7);
  int next = first;  // the step that is loaded next
  auto load = [&](int j, uint32_t take, uint32_t to) {
    const int64_t n = (int64_t)min(next, steps - 1) * kRed;
    if (j < kLw) {
      // rows of W past the last one repeat it: the factor is zero there
      const int nvalid = (int)min((int64_t)kRed, a.N - n);
      const rsrc_t rs = gk::make_rsrc(a.W + n * a.ldw, (uint32_t)(nvalid * a.ldw));
      gk::dma16_if(take, rs, (uint32_t)(min(wrow[j], nvalid - 1) * (int)a.ldw) + wcol[j], 0,
                   to + S::kW + 1024 * (wave + NW * j));
    } else if (SCALED && j == kLoads - 1) {
      const rsrc_t rs = gk::make_rsrc(a.sw, (uint32_t)(4 * a.N));
      gk::dma4_if(take, rs, (uint32_t)(4 * min(n + lane, (int64_t)a.N - 1)), 0,
                  swl0 + (to - lds0) / S::kBytes * (4 * NW * kRed) + 4 * kRed * wave);
    } else {
      const int p = (j - kLw) / kLa, l = (j - kLw) % kLa;
      // columns of the caller's matrix past the last eight repeat them (clear_tail)
      const int over = SCALED ? min(0, 2 * a.N - 16 - (2 * (int)n + achunk)) : 0;
      const rsrc_t rs = gk::make_rsrc(a.P + ((int64_t)p * a.M + m0) * a.pitch,
                                      (uint32_t)mvalid * arow);
      gk::dma16_if(take, rs, aoff[l] + (uint32_t)over, (uint32_t)(2 * n),
                   to + S::kA + p * S::kPlane + 1024 * (wave + NW * l));
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
  v8bf af[2][PLANES * TM];
  constexpr int kU = PLANES * TM;  // products of a fragment of W
  constexpr int kReads = TK + kU + (FORM == kScaledW ? 2 : 0), kProducts = TK * kU;
  constexpr int kPerProduct = (2 * kReads + kProducts - 1) / kProducts;
  const int h = lane >> 5;
  float sc[2][8];
  auto read = [&](int stage, int q, int r) {
    if (FORM == kScaledW && r >= TK + kU) {
      const int x = r - TK - kU;
      const float4 v = *reinterpret_cast<const float4*>(
          swl + (stage * NW + wave) * kRed + 16 * q + 8 * h + 4 * x);
      sc[q & 1][4 * x] = v.x, sc[q & 1][4 * x + 1] = v.y;
      sc[q & 1][4 * x + 2] = v.z, sc[q & 1][4 * x + 3] = v.w;
    } else if (r < TK) {
      const int n = 16 * q + 8 * h + ((lane & 15) >> 1);
      const int c = 2 * (wk * TK + r) + ((lane >> 4) & 1);
      const uint8_t* p = lds + stage * S::kBytes + S::kW + n * BK + 16 * wslot<BK>(n, c) +
                         8 * (lane & 1);
      wraw[q & 1][r] = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
          (__attribute__((address_space(3))) v2i*)p);
    } else {
      const int p = (r - TK) / TM, m = (wm * TM + (r - TK) % TM) * 32 + (lane & 31);
      af[q & 1][r - TK] = *reinterpret_cast<const v8bf*>(lds + stage * S::kBytes + S::kA +
                                                         p * S::kPlane + m * 2 * kRed +
                                                         16 * aslot(m, 2 * q + h));
    }
  };
  // The products of a quarter, and between them the reads of the next one, the
  // loads of a later step, and the conversion of the fragment that the next
  // products take (the next quarter's first in the last of this): a conversion
  // ahead of its products would leave the matrix cores idle.
  v4i wf[2];
  auto convert = [&](int set, int q, int i, int u) {
#pragma unroll
    for (int e = 4 * u / kU; e < 4 * (u + 1) / kU; ++e)
      wf[set][e] = (int)widen_part<FORM == kScaledW>(wraw[q & 1][i], sc[q & 1], e);
  };
  auto quarter = [&](int q, int from, uint32_t take, uint32_t to) {
#pragma unroll
    for (int i = 0; i < TK; ++i) {
      const int set = (q * TK + i) & 1;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int p = i * kU + u;
        acc[i][u % TM] =
            mfma_bf16(__builtin_bit_cast(v8bf, wf[set]), af[q & 1][u], acc[i][u % TM]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = p * kPerProduct; r < (p + 1) * kPerProduct && r < kReads; ++r)
          read(from, (q + 1) & 3, r);
        if (q == 3) {
#pragma unroll
          for (int l = p * kLoads / kProducts; l < (p + 1) * kLoads / kProducts; ++l)
            load(l, take, to);
        }
        if (i + 1 < TK)
          convert(set ^ 1, q, i + 1 < TK ? i + 1 : 0, u);
        else
          convert(set ^ 1, q + 1, 0, u);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

#pragma unroll
  for (int s = 0; s < DEPTH; ++s) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) load(j, s < its, lds0 + s * S::kBytes);
    ++next;
  }
  // the factor's columns from N on, in the last step of all
  const bool tail = FORM == kScaledW && a.N % kRed && first + its == steps;
  auto clear_tail = [&](int stage) {
    for (int i = t; i < BM * 8; i += 64 * NW) {
      const int row = i >> 3, c = i & 7;
      if (c >= a.N % kRed / 8)
        *reinterpret_cast<v4i*>(lds + stage * S::kBytes + S::kA + row * 2 * kRed +
                                16 * aslot(row, c)) = (v4i){0, 0, 0, 0};
    }
    // and the scales that stand there, the last one's copies, which may be infinite
    for (int i = t; i < NW * kRed; i += 64 * NW)
      if (i % kRed >= a.N % kRed) swl[stage * NW * kRed + i] = 0.0f;
    gk::lds_barrier();
  };
  // kScaledA: the factor's rows of step `step`, in place of the caller's; zero from N on
  auto split_rows = [&](int stage, int step) {
    const int row = t / (kRed / 2), n = 2 * (t % (kRed / 2));
    uint8_t* p = lds + stage * S::kBytes + S::kA + row * 2 * kRed + 16 * aslot(row, n >> 3) +
                 2 * (n & 7);
    const uint32_t raw = *reinterpret_cast<const uint32_t*>(p);
    const float2 s = *reinterpret_cast<const float2*>(swl + (stage * NW + wave) * kRed + n);
    const bool in = (int64_t)step * kRed + n < a.N;  // (N is even)
    float v0 = in ? __builtin_bit_cast(float, raw << 16) * s.x : 0.0f;
    float v1 = in ? __builtin_bit_cast(float, raw & 0xffff0000u) * s.y : 0.0f;
#pragma unroll
    for (int i = 0; i < PLANES; ++i) {
      const uint32_t b = bf16_part(v0, i + 1 == PLANES);
      *reinterpret_cast<uint32_t*>(p + i * S::kPlane) = b | bf16_part(v1, i + 1 == PLANES) << 16;
    }
    gk::lds_barrier();
  };
  if (its > 0) {
    wait_vm_if<(DEPTH - 1) * kLoads>(its >= DEPTH);
    gk::lds_barrier();
    if (tail && its == 1) clear_tail(0);
    if constexpr (FORM == kScaledA) split_rows(0, first);
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, 0, r);
#pragma unroll
    for (int u = 0; u < kU; ++u) convert(0, 0, 0, u);
  }
  int buf = 0;
  for (int it = 0; it < its; ++it) {
    const int nbuf = buf == DEPTH - 1 ? 0 : buf + 1;
#pragma unroll
    for (int q = 0; q < 3; ++q) quarter(q, buf, 0, 0);
    wait_vm_if<(DEPTH - 2) * kLoads>(it + DEPTH - 1 < its);
    gk::lds_barrier();
    if (tail && it + 2 == its) clear_tail(nbuf);
    if (FORM == kScaledA && it + 1 < its) split_rows(nbuf, first + it + 1);
    quarter(3, nbuf, it + DEPTH < its, lds0 + buf * S::kBytes);
    ++next;
    buf = nbuf;
  }

#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int64_t m = m0 + (wm * TM + j) * 32 + (lane & 31);
    if (m >= a.M) continue;
#pragma unroll
    for (int i = 0; i < TK; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int k = k0 + (wk * TK + i) * 32 + 8 * g + 4 * h;
        float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                               acc[i][j][4 * g + 3]);
        if (!a.acc) {
          if (k < a.K) put_result(a.out, m, k, a.K, v);
          continue;
        }
        if (k >= a.kp) continue;
        float4* p = reinterpret_cast<float4*>(a.acc + ((int64_t)split * a.M + m) * a.kp + k);
        if (a.add) {
          const float4 o = *p;
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        *p = v;
      }
  }
}

// A[m, n] = dY[m, n] * sw[n] as `planes` bf16 matrices, zero from column N to
// the pitch.  A workgroup takes 2048 columns of ROWS rows, a thread eight of each:
// four rows where there are many (2048 x 12288 bf16: 18.4 us, one row 54), one
// where few would leave the chip idle (77 x 1037 f32: 5 us, four rows 9).
template <int TYPE, int ROWS, bool ONE>
__global__ __launch_bounds__(256) void planes_kernel(const void* dY, int64_t lddy, bool wide,
                                                     const float* sw, uint16_t* P, int64_t pitch,
                                                     int planes, int M, int N) {
  const int64_t m0 = (blockIdx.y + (int64_t)gridDim.y * blockIdx.z) * ROWS;
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (n >= pitch) return;  // the pitch is a multiple of 64
  float f[8], v[ROWS][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = n + e < N ? sw[n + e] : 0.0f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t at = min(m0 + r, (int64_t)M - 1) * lddy + n;
    if constexpr (TYPE == GEMMQ_F32) {
      float a[4], b[4];
      load_values<TYPE, 4>(dY, at, N - n, wide, a);
      load_values<TYPE, 4>(dY, at + 4, N - n - 4, wide, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[r][e] = a[e], v[r][e + 4] = b[e];
    } else {
      load_values<TYPE, 8>(dY, at, N - n, wide, v[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (m0 + r >= M) return;
    uint16_t* to = P + (m0 + r) * pitch + n;
    // columns from N on are zero, not the product of what is read there with zero
#pragma unroll
    for (int e = 0; e < 8; ++e) v[r][e] = n + e < N ? v[r][e] * f[e] : 0.0f;
    if constexpr (ONE) {
      *reinterpret_cast<uint4*>(to) =
          make_uint4(bf16_bits(v[r][0]) | bf16_bits(v[r][1]) << 16,
                     bf16_bits(v[r][2]) | bf16_bits(v[r][3]) << 16,
                     bf16_bits(v[r][4]) | bf16_bits(v[r][5]) << 16,
                     bf16_bits(v[r][6]) | bf16_bits(v[r][7]) << 16);
      continue;
    }
    for (int p = 0; p < planes; ++p) {
      uint32_t b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        b[e] = bf16_part(v[r][2 * e], p + 1 == planes);
        b[e] |= bf16_part(v[r][2 * e + 1], p + 1 == planes) << 16;
      }
      *reinterpret_cast<uint4*>(to + (int64_t)p * M * pitch) = make_uint4(b[0], b[1], b[2], b[3]);
    }
  }
}

// The ranges' sums added up, always in the same order: a thread takes four
// columns of a row and one of GROUPS stretches of the ranges, eight of them at a
// time, and the stretches are added through LDS.
template <int GROUPS>
__global__ __launch_bounds__(256) void finish_kernel(const float* acc, int64_t kp, int splits,
                                                     GradOut out, int M, int K) {
  constexpr int kQuads = 256 / GROUPS;
  __shared__ float4 part[GROUPS > 1 ? 256 : 1];
  const int64_t m = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
  if (m >= M) return;  // all of the workgroup
  const int quad = threadIdx.x % kQuads, group = threadIdx.x / kQuads;
  const int k = (blockIdx.x * kQuads + quad) * 4;
  const int per = (splits + GROUPS - 1) / GROUPS;
  const int first = group * per, end = min(first + per, splits);
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (k < K) {
    for (int s = first; s < end; s += 8) {
      float4 w[8];
      // a row of acc is whole to its pitch, a multiple of 4
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = *reinterpret_cast<const float4*>(acc + ((int64_t)min(s + e, end - 1) * M + m) * kp +
                                                k);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (s + e < end) v = make_float4(v.x + w[e].x, v.y + w[e].y, v.z + w[e].z, v.w + w[e].w);
    }
  }
  if constexpr (GROUPS > 1) {
    part[threadIdx.x] = v;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const float4 w = part[g * kQuads + quad];
      v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
    }
  }
  if (k < K) put_result(out, m, k, K, v);
}

// A tile, and by the factor's planes (1 to 3) the time of a step (us) on a compute
// unit that works on one, two or three such workgroups at a time, 0 where its LDS
// holds fewer or there is no such tile.
struct Tile {
  int bk, bm;
  float step[3][3];
};
constexpr Tile kTiles[] = {
    {256, 256, {{1.5f}}},
    {256, 128, {{1.0f, 1.7f}, {1.5f}, {2.15f}}},
    {128, 128, {{0.69f, 1.05f}, {0.9f, 1.55f}, {1.25f}}},
    {128, 64, {{0.56f, 0.77f, 1.1f}, {0.67f, 1.0f}, {0.8f, 1.3f}}},
    {128, 32, {{0.5f, 0.6f}, {0.55f, 0.75f}, {0.62f, 0.85f}}}};
constexpr int kCUs = 256, kMaxThreads = 512;

int64_t tiles(const Tile& c, int M, int K) { return ceil_div(M, c.bm) * ceil_div(K, c.bk); }

}  // namespace

// The tile and the number of ranges with the least estimated time: rounds of the
// chip, each of its range's steps and 3 us around them, and for partial sums their
// passage through memory (4.5 TB/s) and a launch's 3 (M = 1 over 364 x 2724 took 12 us
// as one range and 16 as six).  Measured (us, with the sums' launch; the best number
// of ranges for each tile in the order of kTiles, the one taken in brackets):
//   one plane   M 16 N 4096 K 4096      -      -      -     11.8 [11.1]
//               M 128 N 12288 K 4096    40     33   [30]    32    33
//               M 200 N 2048 K 2048     23     18     15   [14]
//               M 512 N 12288 K 4096    66   [65]     67    85
//               M 2048 N 4096 K 4096    88   [74]     77   107
//               M 2048 N 12288 K 4096 [193]   202    218   309
//   two         M 1024 N 4096 K 4096     -     69   [67]    73
//   three       M 1500 N 2560 K 5008     -   [92]    114   118
//               M 64 N 12288 K 4096      -     38     41   [30]   31
// The two widest would be more than half empty up to 128 tokens, the lowest reads W
// too often beyond; up to 8 it is the fastest of the three.  A range has at least one step.
GradSplit grad_split(int M, int N, int K, int planes, bool whole) {
  const int64_t steps = ceil_div(N < 1 ? 1 : N, kRed);
  GradSplit best{0, 0};
  double least = 0.0;
  for (int i = M <= 8 ? 4 : M <= 128 ? 2 : 0; i <= (M <= 128 ? 4 : 3); ++i) {
    const float* step = kTiles[i].step[planes - 1];
    if (!(step[0] > 0.0f)) continue;
    const int64_t n = tiles(kTiles[i], M, K);
    // one range, or as many as fill the chip with one, two or three workgroups
    for (int f = 0; f <= 3; ++f) {
      if (f > 0 && !(step[f - 1] > 0.0f)) break;
      int64_t s = f == 0 ? 1 : kCUs * f / n;
      if (s > steps) s = steps;
      if (s < 1) continue;
      int r = 1;
      while (r < 3 && step[r] > 0.0f && n * s > kCUs * r) ++r;
      double t = (double)ceil_div(n * s, kCUs * r) *
                 ((double)ceil_div(steps, s) * step[r - 1] + 3.0);
      if (s > 1 || !whole) t += 3.0 + (double)s * M * K * 8e-6 / 4.5;
      if (best.splits == 0 || t < least) {
        best = GradSplit{i, (int)s};
        least = t;
      }
    }
  }
  return best;
}

bool grad_fits(const GradSplit& s, int M, int K) {
  return grid_fits(tiles(kTiles[s.tile], M, K) * s.splits, kMaxThreads);
}

int launch_grad(const GradArgs& a, hipStream_t st) {
  const Tile& c = kTiles[a.tile];
  const uint32_t mt = (uint32_t)ceil_div(a.M, c.bm), kt = (uint32_t)ceil_div(a.K, c.bk);
  const int64_t n = (int64_t)mt * kt * a.splits;
  if (!grid_fits(n, kMaxThreads)) return -1;
  const dim3 grid((uint32_t)n);
  const auto run = [&](auto kernel, int threads) { kernel<<<grid, threads, 0, st>>>(a, kt, mt); };
  // with sw: up to 128 tokens, in the lower three tiles; two planes up to 8, in the lowest
  switch (a.tile) {
    case 0: run(grad_kernel<256, 256, 4, 2, 3, 1, kPlanes>, 512); break;
    case 1:
      a.planes == 1   ? run(grad_kernel<256, 128, 4, 2, 2, 1, kPlanes>, 512)
      : a.planes == 2 ? run(grad_kernel<256, 128, 4, 2, 3, 2, kPlanes>, 512)
                      : run(grad_kernel<256, 128, 4, 2, 2, 3, kPlanes>, 512);
      break;
    case 2:
      a.sw            ? run(grad_kernel<128, 128, 2, 2, 3, 1, kScaledW>, 256)
      : a.planes == 1 ? run(grad_kernel<128, 128, 2, 2, 3, 1, kPlanes>, 256)
      : a.planes == 2 ? run(grad_kernel<128, 128, 2, 2, 2, 2, kPlanes>, 256)
                      : run(grad_kernel<128, 128, 2, 2, 2, 3, kPlanes>, 256);
      break;
    case 3:
      a.sw            ? run(grad_kernel<128, 64, 2, 2, 3, 1, kScaledW>, 256)
      : a.planes == 1 ? run(grad_kernel<128, 64, 2, 2, 3, 1, kPlanes>, 256)
      : a.planes == 2 ? run(grad_kernel<128, 64, 2, 2, 3, 2, kPlanes>, 256)
                      : run(grad_kernel<128, 64, 2, 2, 2, 3, kPlanes>, 256);
      break;
    default:
      a.sw            ? a.planes == 1 ? run(grad_kernel<128, 32, 4, 1, 3, 1, kScaledW>, 256)
                                      : run(grad_kernel<128, 32, 4, 1, 3, 2, kScaledA>, 256)
      : a.planes == 1 ? run(grad_kernel<128, 32, 4, 1, 3, 1, kPlanes>, 256)
      : a.planes == 2 ? run(grad_kernel<128, 32, 4, 1, 3, 2, kPlanes>, 256)
                      : run(grad_kernel<128, 32, 4, 1, 3, 3, kPlanes>, 256);
  }
  return 0;
}

int launch_planes(int type, const void* dY, int64_t lddy, const float* sw, uint16_t* P,
                  int64_t pitch, int planes, int M, int N, hipStream_t st) {
  // (bf16 in two planes: up to eight rows)
  const bool many = M * pitch >= (int64_t)1 << 22 && (type != GEMMQ_BF16 || planes == 1);
  const bool wide = wide_rows(dY, lddy, type);
  const dim3 grid = rows_grid(ceil_div(pitch, 2048), many ? ceil_div(M, 4) : M);
  const auto run = [&](auto kernel) {
    kernel<<<grid, 256, 0, st>>>(dY, lddy, wide, sw, P, pitch, planes, M, N);
  };
  if (type == GEMMQ_F32)
    many ? run(planes_kernel<GEMMQ_F32, 4, false>) : run(planes_kernel<GEMMQ_F32, 1, false>);
  else if (type == GEMMQ_F16)
    many ? run(planes_kernel<GEMMQ_F16, 4, false>) : run(planes_kernel<GEMMQ_F16, 1, false>);
  else if (planes == 1)
    many ? run(planes_kernel<GEMMQ_BF16, 4, true>) : run(planes_kernel<GEMMQ_BF16, 1, true>);
  else  // few rows
    run(planes_kernel<GEMMQ_BF16, 1, false>);
  return 0;
}

int launch_finish(const float* acc, int64_t kp, int splits, const GradOut& out, int M, int K,
                  hipStream_t st) {
  // many ranges (few rows: the chip is otherwise idle) are read by four threads a column
  if (splits >= 16)
    finish_kernel<4><<<rows_grid(ceil_div(K, 256), M), 256, 0, st>>>(acc, kp, splits, out, M, K);
  else
    finish_kernel<1><<<rows_grid(ceil_div(K, 1024), M), 256, 0, st>>>(acc, kp, splits, out, M, K);
  return 0;
}

}  // namespace i8
}  // namespace gemmq
