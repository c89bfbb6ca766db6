// i8_common.h -- device pieces the int8 kernels share.
#pragma once

#include "gemm_common.h"
#include "i8.h"

namespace gemmq {
namespace i8 {

using gk::rsrc_t;
using gk::v16f;
using gk::v16i;
using gk::v4i;

typedef __bf16 bf16_t;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// what a product's kernel does with its sums
enum Epilogue { kLinear, kLoss, kFactor, kAct, kGate };

// f32 -> the type's 16 bits, round to nearest even
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (bf16_t)v);
}
// what that rounding leaves of v, exactly
__device__ __forceinline__ float bf16_rest(float v) {
  return v - __builtin_bit_cast(float, bf16_bits(v) << 16);
}
__device__ __forceinline__ uint32_t f16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}

__device__ __forceinline__ float load_as_f32(const void* p, int64_t i, int type) {
  if (type == GEMMQ_F32) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  if (type == GEMMQ_BF16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  return (float)__builtin_bit_cast(_Float16, b);
}

__device__ __forceinline__ void store_as(void* p, int64_t i, int type, float v) {
  if (type == GEMMQ_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] = (uint16_t)(type == GEMMQ_BF16 ? bf16_bits(v) : f16_bits(v));
}

// four consecutive values of a row from element i: at once where `wide` says that
// the address allows it and all four are inside, else those of the first `count`
__device__ __forceinline__ void store4_as(void* p, int64_t i, int type, bool wide, int count,
                                          float v0, float v1, float v2, float v3) {
  if (wide && count >= 4) {
    if (type == GEMMQ_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v0, v1, v2, v3);
    } else {
      uint2 b;
      if (type == GEMMQ_BF16)
        b = make_uint2(bf16_bits(v0) | bf16_bits(v1) << 16, bf16_bits(v2) | bf16_bits(v3) << 16);
      else
        b = make_uint2(f16_bits(v0) | f16_bits(v1) << 16, f16_bits(v2) | f16_bits(v3) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = b;
    }
    return;
  }
  if (count > 0) store_as(p, i, type, v0);
  if (count > 1) store_as(p, i + 1, type, v1);
  if (count > 2) store_as(p, i + 2, type, v2);
  if (count > 3) store_as(p, i + 3, type, v3);
}

// the values of two 16-bit halves of a word, bf16 or f16
__device__ __forceinline__ float2 halves(uint32_t w, int type) {
  if (type == GEMMQ_BF16)
    return make_float2(__builtin_bit_cast(float, w << 16),
                       __builtin_bit_cast(float, w & 0xffff0000u));
  return make_float2((float)__builtin_bit_cast(_Float16, (uint16_t)w),
                     (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16)));
}
// two values as such a word, rounded
__device__ __forceinline__ uint32_t two_bits(float a, float b, int type) {
  return type == GEMMQ_BF16 ? bf16_bits(a) | bf16_bits(b) << 16 : f16_bits(a) | f16_bits(b) << 16;
}

// four consecutive values of a row from element i, as store4_as; zero past `count`
__device__ __forceinline__ void load4_as(const void* p, int64_t i, int type, bool wide, int count,
                                         float (&v)[4]) {
  if (wide && count >= 4) {
    if (type == GEMMQ_F32) {
      const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
      const float2 lo = halves(x.x, type), hi = halves(x.y, type);
      v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = e < count ? load_as_f32(p, i + e, type) : 0.0f;
}

// The next bf16 of v's expansion, its top 16 bits, and what is left of v: both
// exact, so three of them hold all 24 bits of an f32 (the last one is rounded,
// which matters for two).  An infinity or a NaN is its own only part, with the
// quiet bit set so that a NaN whose set bits are all in the low half stays one.
__device__ __forceinline__ uint32_t bf16_part(float& v, bool last) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  if ((b & 0x7f800000u) == 0x7f800000u) {
    v = 0.0f;
    return (b >> 16) | ((b & 0x7fffffu) ? 0x40u : 0u);
  }
  if (last) return bf16_bits(v);
  v -= __builtin_bit_cast(float, b & 0xffff0000u);
  return b >> 16;
}

// vmcnt(N) where the wave-uniform `most` holds, else vmcnt(0); without a branch
// that the compiler sees
template <int N>
__device__ __forceinline__ void wait_vm_if(bool most) {
  static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit field");
  if constexpr (N == 0) {
    gk::wait_vm<0>();
  } else {
    const uint32_t t = __builtin_amdgcn_readfirstlane((uint32_t)most);
    asm volatile(
        "s_cmp_eq_u32 %0, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(%1)\n\ts_branch 2f\n"
        "1:\ts_waitcnt vmcnt(0)\n2:" ::"s"(t),
        "i"(N)
        : "memory", "scc");
  }
}

// v = sw dot as the epilogues have it, in f32 from dot in f32, and what its two roundings
// leave: sw dot = v + left, to f32 precision of left.  (|dot| <= 2^31 - 2^14, so dot in f32
// is an int32 too, and dot less it, at most 64, an f32.)
__device__ __forceinline__ float scaled(int dot, float sw, float& left) {
  const float d = (float)dot, v = d * sw;
  left = fmaf((float)(dot - (int)d), sw, fmaf(d, sw, -v));
  return v;
}

// exp(z - lse) - 1 at the target, z = sx sw dot.  Near certainty the difference is
// small against z, whose rounding (half a step of sw dot) would be most of it: the
// product's remainder is carried along, and nothing is subtracted from 1.
__device__ __forceinline__ float target_factor(int dot, float sw, float sx, float lse) {
  float left;
  const float v = scaled(dot, sw, left);
  return expm1f(fmaf(left, sx, fmaf(v, sx, -lse)));
}

// f[0..3] as `planes` matrices of bf16 parts, `plane` elements apart
__device__ __forceinline__ void store_planes(uint16_t* p, int64_t plane, int planes, float (&f)[4]) {
  if (planes == 1) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_bits(f[0]) | bf16_bits(f[1]) << 16,
                                              bf16_bits(f[2]) | bf16_bits(f[3]) << 16);
    return;
  }
  for (int i = 0; i < planes; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = bf16_part(f[e], i + 1 == planes);
    *reinterpret_cast<uint2*>(p + i * plane) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  }
}

// the first `keep` bytes of v, the others zero
__device__ __forceinline__ v4i keep_bytes(v4i v, int keep) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int b = keep - 4 * w;
    v[w] = b >= 4 ? v[w] : b <= 0 ? 0 : v[w] & ((1 << (8 * b)) - 1);
  }
  return v;
}

// ---- the row quantizer's arithmetic (gemmq_quantize_i8)

// |x| as an unsigned integer: ordered as the values, infinity above every finite
// one and NaN above infinity, so that a maximum shows either.
__device__ __forceinline__ uint32_t abs_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
}
// a row's scale from its largest abs_bits: NaN where the row is not finite
__device__ __forceinline__ float scale_of(uint32_t top) {
  return top < 0x7f800000u ? __builtin_bit_cast(float, top) / 127.0f : __builtin_nanf("");
}
// x / s to the nearest integer, ties to even, within [-127, 127], for a row with a
// finite s > 0 and inv = 1 / s.  x * inv is within 2^-23 |x / s| < 2 10^-5 of the
// quotient, and the rounded quotient within 10^-5: unless x * inv lies within 10^-4
// of a tie (or inv is infinite), all three round to the same integer, and the
// division, half of the quantizer's arithmetic, is left out.
__device__ __forceinline__ float quantized(float x, float s, float inv) {
  const float t = x * inv;
  float q = rintf(t);
  if (!(fabsf(t - q) < 0.4999f)) q = rintf(x / s);
  return __builtin_amdgcn_fmed3f(q, -127.0f, 127.0f);
}

// 16 bytes, with ONCE as those of a stream that nothing reads or writes again soon
template <bool ONCE>
__device__ __forceinline__ uint4 load_line(const void* p) {
  typedef uint32_t Line __attribute__((ext_vector_type(4)));
  if constexpr (!ONCE) return *static_cast<const uint4*>(p);
  const Line v = __builtin_nontemporal_load(static_cast<const Line*>(p));
  return make_uint4(v.x, v.y, v.z, v.w);
}
template <bool ONCE>
__device__ __forceinline__ void store_line(void* p, uint4 w) {
  typedef uint32_t Line __attribute__((ext_vector_type(4)));
  if constexpr (ONCE)
    __builtin_nontemporal_store(Line{w.x, w.y, w.z, w.w}, static_cast<Line*>(p));
  else
    *static_cast<uint4*>(p) = w;
}

// 16 bytes of a row from element i, zero from element `end` of the row on (`left`
// values are left before it); at once where the row allows 16-byte loads and all
// are there
template <int TYPE, bool ONCE = false>
__device__ __forceinline__ uint4 load_raw(const void* p, int64_t i, int64_t left, bool wide) {
  constexpr int V = TYPE == GEMMQ_F32 ? 4 : 8;
  uint32_t u[4] = {0, 0, 0, 0};
  if constexpr (TYPE == GEMMQ_F32) {
    const uint32_t* x = static_cast<const uint32_t*>(p) + i;
    if (wide && left >= V) return load_line<ONCE>(x);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < left) u[e] = x[e];
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(p) + i;
    if (wide && left >= V) return load_line<ONCE>(x);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < left) u[e >> 1] |= (uint32_t)x[e] << (16 * (e & 1));
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// the V values of 16 bytes as f32
template <int TYPE, int V>
__device__ __forceinline__ void unpack(uint4 w, float (&v)[V]) {
  static_assert(V == (TYPE == GEMMQ_F32 ? 4 : 8), "16 bytes");
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < V; ++e) {
    if constexpr (TYPE == GEMMQ_F32) {
      v[e] = __builtin_bit_cast(float, u[e]);
    } else if constexpr (TYPE == GEMMQ_BF16) {
      v[e] = __builtin_bit_cast(float, e & 1 ? u[e >> 1] & 0xffff0000u : u[e >> 1] << 16);
    } else {
      v[e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[e >> 1] >> (16 * (e & 1))));
    }
  }
}

template <int TYPE, int V>
__device__ __forceinline__ void load_values(const void* p, int64_t i, int64_t left, bool wide,
                                            float (&v)[V]) {
  unpack<TYPE, V>(load_raw<TYPE>(p, i, left, wide), v);
}

// how many values of a row 16 bytes hold
template <int TYPE>
constexpr int kValues = TYPE == GEMMQ_F32 ? 4 : 8;

// f32 values as 16 bytes of a row, rounded to its type
template <int TYPE, int V>
__device__ __forceinline__ uint4 pack(const float (&v)[V]) {
  static_assert(V == kValues<TYPE>, "16 bytes");
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (TYPE == GEMMQ_F32)
      u[i] = __builtin_bit_cast(uint32_t, v[i]);
    else if constexpr (TYPE == GEMMQ_BF16)
      u[i] = bf16_bits(v[2 * i]) | bf16_bits(v[2 * i + 1]) << 16;
    else
      u[i] = f16_bits(v[2 * i]) | f16_bits(v[2 * i + 1]) << 16;
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// 16 bytes to a row from element i on, those of its first `left` values
template <int TYPE, bool ONCE = false>
__device__ __forceinline__ void store_raw(void* p, int64_t i, int left, bool wide, uint4 w) {
  constexpr int V = kValues<TYPE>;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (TYPE == GEMMQ_F32) {
    uint32_t* to = static_cast<uint32_t*>(p) + i;
    if (wide && left >= V) {
      store_line<ONCE>(to, w);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) to[e] = u[e];
    }
  } else {
    uint16_t* to = static_cast<uint16_t*>(p) + i;
    if (wide && left >= V) {
      store_line<ONCE>(to, w);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < left) to[e] = (uint16_t)(u[e >> 1] >> (16 * (e & 1)));
    }
  }
}

// V quantized values as bytes, zero in a row whose scale is 0 or NaN
template <int V>
__device__ __forceinline__ void quantize_values(const float (&v)[V], float s, float inv,
                                                uint32_t (&q)[V / 4]) {
#pragma unroll
  for (int w = 0; w < V / 4; ++w) {
    uint32_t b[4];
    // 1.5 2^23 + q holds q's two's complement in its low bits
#pragma unroll
    for (int e = 0; e < 4; ++e)
      b[e] = __builtin_bit_cast(uint32_t, quantized(v[4 * w + e], s, inv) + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    q[w] = s > 0.0f ? lo | hi : 0u;
  }
}

// ---- sums and maxima over a wave, in every lane: within rows of 16 lanes by moves between
// lanes, across them by exchanged halves (through ds_bpermute a sum in f64 took 12 trips to LDS)

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xf, 0xf, true);
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

// op(own value, the other lane's), for lanes 1, 2, 4, 8, 16 and 32 apart (4 and 8 as mirror
// images: the lanes of what is joined already hold the same value)
template <int CTRL, class Op>
__device__ __forceinline__ double join_lanes(double v, Op op) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t o = (uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b);
  return op(v, __builtin_bit_cast(double, o));
}
__device__ __forceinline__ double wave_sum(double v) {
  auto add = [](double a, double b) { return a + b; };
  v = join_lanes<kXor1>(v, add);
  v = join_lanes<kXor2>(v, add);
  v = join_lanes<kHalfMirror>(v, add);
  v = join_lanes<kMirror>(v, add);
  auto halves = [](auto lo, auto hi) {
    return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) +
           __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  };
  uint64_t b = __builtin_bit_cast(uint64_t, v);
  v = halves(__builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false),
             __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
  b = __builtin_bit_cast(uint64_t, v);
  return halves(
      __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false),
      __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// the sum over the workgroup of T threads of v[0..N), in every thread and in a fixed
// order; `at`: N * T / 64 doubles of LDS that nothing else uses
template <int T, int N>
__device__ __forceinline__ void sum_all(double (&v)[N], double* at, int t) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if ((t & 63) == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) at[N * (t >> 6) + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = at[i];
#pragma unroll
  for (int w = 1; w < T / 64; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += at[N * w + i];
}

// Workgroup index -> position in the work list such that each of the eight XCDs
// (consecutive workgroups go to consecutive XCDs) takes one contiguous stretch
// of it, and neighbours in the list share an L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t total) {
  const uint32_t xcd = id & 7, at = id >> 3, per = total >> 3, more = total & 7;
  return xcd * per + (xcd < more ? xcd : more) + at;
}

}  // namespace i8
}  // namespace gemmq
