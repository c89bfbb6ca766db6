// i8_check.h -- the checks of arguments that the int8 half's entry points share.
#pragma once

#include "abi_util.h"
#include "gemmq_i8.h"
#include "i8.h"

namespace gemmq {
namespace i8 {

constexpr int64_t kMaxPitchElems = (int64_t)1 << 40;  // keeps element offsets below 2^63

inline bool known(int type) { return type == GEMMQ_F32 || type == GEMMQ_BF16 || type == GEMMQ_F16; }

inline int check_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0) return GEMMQ_E_INVALID_ARG;
  if (K < 1 || K > GEMMQ_I8_MAX_K || M > GEMMQ_I8_MAX_ROWS || N > GEMMQ_I8_MAX_ROWS)
    return GEMMQ_E_SHAPE;
  return GEMMQ_OK;
}

// an int8 matrix with its scales
inline int check_i8(const void* p, int64_t ld, const void* s, int64_t K) {
  if (!p || !s) return GEMMQ_E_INVALID_ARG;
  if (ld < K || ld > GEMMQ_I8_MAX_PITCH) return GEMMQ_E_SHAPE;
  if (ld % 16 != 0 || !aligned(p, 16) || !aligned(s, 4)) return GEMMQ_E_ALIGNMENT;
  return GEMMQ_OK;
}

// a matrix of element type `type`
inline int check_rows(int type, const void* p, int64_t ld, int64_t width) {
  if (!known(type) || !p) return GEMMQ_E_INVALID_ARG;
  if (ld < width || ld > kMaxPitchElems) return GEMMQ_E_SHAPE;
  if (!aligned(p, (uintptr_t)type_bytes(type))) return GEMMQ_E_ALIGNMENT;
  return GEMMQ_OK;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return GEMMQ_E_INVALID_ARG;
  return aligned(ws, 16) ? GEMMQ_OK : GEMMQ_E_ALIGNMENT;
}

// Whether a row of one matrix shares memory with a row of the other, for the few rows of the
// products that quantize X in their own launch: each of its workgroups reads all of X while
// others already store results, so results in X's place need the launches apart.
struct Span {
  const void* p;  // null: no matrix
  int64_t pitch, width;  // bytes
};
inline Span span(int type, const void* p, int64_t ld, int64_t width) {
  return {p, ld * type_bytes(type), width * type_bytes(type)};
}
inline bool share_memory(const Span& a, const Span& b, int64_t M) {
  if (!a.p || !b.p) return false;
  for (int64_t i = 0; i < M; ++i)
    for (int64_t j = 0; j < M; ++j) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(a.p) + i * a.pitch;
      const uintptr_t y = reinterpret_cast<uintptr_t>(b.p) + j * b.pitch;
      if (x < y + b.width && y < x + a.width) return true;
    }
  return false;
}

inline size_t align_up(int64_t v, int64_t a) { return (size_t)((v + a - 1) / a * a); }

}  // namespace i8
}  // namespace gemmq
