// i8_sample.hip -- one token a row from its logits (gemmq_sample): temperature, top-k,
// top-p, min-p and a given random number, without sorting the vocabulary.
//
// The tokens stand in descending order of their logits (equal ones by index), and every
// limit keeps a prefix of that order, so all that is asked for are places in it: where the
// count reaches k, where the sum of the weights reaches p of what that leaves, where the
// weights fall below min_p, and where the sum passes u of what all of them leave.  A
// histogram over the distance from the largest logit (a function of the logit that never
// rises, so its bins are in that order) says which bins' tokens matter, and only those are
// gathered and sorted:
//   with a k of at most kListedK, all down to the k-th, by a histogram of counts: only those
//   tokens' weights are ever computed;
//   else by a histogram of weights, the bins that the places lie in.  Bounds of the sum that
//   one limit leaves give the next one a range of bins.
//
// A row of up to 32768 f32 or 65536 16-bit logits is held by one workgroup's registers, and one
// launch does all of it (whole_kernel).  Longer ones, and in some cases (is_whole) shorter ones,
// are spread over as many workgroups as fill the chip, in four launches: the rows' largest
// logits; the histograms; the gathering; the draw.
//
// Weights are integers, e = exp((z - max) / t) in units of 2^-bits: their sums are exact, so
// atomics may add them in any order.  e is computed in f64, to 10^-14: with f32's 10^-7 one
// row in a few hundred of a flat distribution would draw the neighbour of the token that
// the definition draws.
#include <float.h>

#include "i8_block.h"
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

typedef unsigned long long u64;

constexpr int kBins = 2048;   // of a row's histogram
constexpr int kList = 4096;   // tokens that are sorted; a row whose bins hold more is searched
                              // by its logits' bits instead (as where all logits are equal)
constexpr int kListedK = kList / 2;
constexpr int kThreads = 256; // of a workgroup that goes through a part of a row
constexpr int kDraw = 512;    // of one that draws

// ordered as the values are, -0 as +0; of finite values and infinities
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, key ^ ((uint32_t)((int32_t)~key >> 31) | 0x80000000u));
}
// a token in a list: descending order is the order of the tokens
__device__ __forceinline__ u64 entry_of(float z, uint32_t index) {
  return (u64)key_of(z) << 32 | (uint32_t)~index;
}

// A workgroup's part of a row in registers: up to 16384 logits, P 16-byte pieces a thread.
// Launches 1 to 3 load it whole before they look at anything else, so that what they work out
// of the row first overlaps the loads.
constexpr int kMostOfARow = 16384;
template <int TYPE, int T = kThreads, int P = kMostOfARow / (kThreads * kValues<TYPE>)>
struct Part {
  static constexpr int V = kValues<TYPE>, kSpan = V * T;
  uint4 raw[P];
  int begin, end, t;

  // logits [first, past) of row m, at most P * kSpan of them
  __device__ __forceinline__ Part(const SampleArgs& a, int64_t m, int first, int past, int thread) {
    t = thread;
    begin = first;
    end = past;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int n0 = begin + kSpan * i, n = n0 + V * t;
      if (n0 >= end) break;
      // (the same way in all lanes wherever the piece is whole)
      if (a.wide && n0 + kSpan <= end)
        raw[i] = load_raw<TYPE>(a.Z, m * a.ldz + n, V, true);
      else
        raw[i] = load_raw<TYPE>(a.Z, m * a.ldz + n, end - n, a.wide);
    }
    asm volatile("" ::: "memory");  // or the compiler moves each load to its use
  }
  // piece(v, index of v[0]) for each, with -inf, which counts nowhere, past the end
  template <class Piece>
  __device__ __forceinline__ void pieces(Piece piece) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int n0 = begin + kSpan * i, n = n0 + V * t;
      if (n0 >= end) break;
      float v[V];
      unpack<TYPE, V>(raw[i], v);
      if (n0 + kSpan > end) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (n + e >= end) v[e] = -__builtin_inff();
      }
      piece(v, n);
    }
  }
  // each(z, index)
  template <class Each>
  __device__ __forceinline__ void logits(Each each) const {
    pieces([&](const float(&v)[V], int n) {
#pragma unroll
      for (int e = 0; e < V; ++e) each(v[e], n + e);
    });
  }
};

// the workgroup's part of its row
template <int TYPE>
__device__ __forceinline__ Part<TYPE> part_of(const SampleArgs& a, int64_t m, int t) {
  const int begin = blockIdx.x * a.chunk;
  return Part<TYPE>(a, m, begin, min(begin + a.chunk, a.N), t);
}

// each(z, index) for a whole row, by a workgroup of T threads
template <int TYPE, int T, class Each>
__device__ __forceinline__ void for_row(const SampleArgs& a, int64_t m, int t, Each each) {
  constexpr int V = kValues<TYPE>;
  for (int n = V * t; n < a.N; n += V * T) {
    float v[V];
    load_values<TYPE, V>(a.Z, m * a.ldz + n, a.N - n, a.wide, v);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (n + e < a.N) each(v[e], n + e);
  }
}

struct Limits {
  int k;      // 0: none
  double p;   // 1: none
  double y;   // log2 of min_p; below -100: none
  double u;
};

__device__ __forceinline__ Limits limits_of(const SampleArgs& a, int64_t m) {
  Limits l;
  const int k = a.top_k ? a.top_k[m] : 0;
  l.k = k > 0 && k < a.N ? k : 0;
  const float p = a.top_p ? a.top_p[m] : 1.0f, q = a.min_p ? a.min_p[m] : 0.0f;
  l.p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;
  l.y = q > 0.0f ? log2((double)fminf(q, 1.0f)) : -1000.0;
  const float u = a.u[m];
  l.u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
  return l;
}

// What the launches after the first know of a row, from the parts' results and the row's
// settings: worked out by the second one's workgroups, and kept for the others
struct Row {
  Limits l;
  double rate;  // log2 e / temperature
  float top;    // the largest logit
  float floor;  // tokens below it count nowhere: their weights are zero, or min_p is the only
                // limit to a sum and takes them out
  float least;  // min_p's limit: kept from here on
  float scale;  // bins per unit of distance
  bool bad, greedy;
  // the kinds of rows: down to the k-th token, or by sums
  __device__ bool listed() const { return l.k > 0 && l.k <= kListedK; }
  __device__ bool by_p() const { return l.p > 0.0 && l.p < 1.0; }
  __device__ bool by_q() const { return least > floor; }
  // Rows of which all tokens (from min_p on) are kept: one is nearly certain where the others'
  // sum is next to nothing, which the logarithm of its share is then as exact as, so that
  // sum is taken in f64 too (a unit for each of 150000 tokens is 4 10^-9).  Limits that keep
  // more than the first token leave a sum that integers hold, or a list to add up.
  __device__ bool exact() const { return l.k == 0 && l.p >= 1.0; }
};

// places that are lo at least and not at hi (a NaN: without an end), some of them none
struct Ranges {
  float lo[4], hi[4];
  bool one;  // from the first place on
};
struct RowAndRanges {
  Row row;
  Ranges ranges;
};
__device__ __forceinline__ RowAndRanges* rows_of(const SampleArgs& a) {
  return static_cast<RowAndRanges*>(a.rows);
}

// log2 of a token's weight relative to the largest
__device__ __forceinline__ double log2_weight(const Row& r, float z) {
  return ((double)z - (double)r.top) * r.rate;
}
// the distance from the largest logit in bins (0 <= ; infinite, or with a scale of 0 NaN, where
// z is -inf), which never rises with z, and for z >= r.floor the bin: the last one holds all that
// lies behind it too
__device__ __forceinline__ float place_of(const Row& r, float z) { return (r.top - z) * r.scale; }
__device__ __forceinline__ int bin_of(const Row& r, float z) {
  return (int)fminf(place_of(r, z), (float)(kBins - 1));
}
// places of bins lo .. hi: from lo to below past(hi), which for the last is a NaN: no place is
// behind it, nor is an infinite one, of a distance past f32
__device__ __forceinline__ float past(int hi) {
  return hi == kBins - 1 ? __builtin_nanf("") : (float)(hi + 1);
}

__device__ __forceinline__ void join(SamplePart& s, const SamplePart& o) {
  s.top = fmaxf(s.top, o.top);
  s.low = fminf(s.low, o.low);
  s.bad |= o.bad;
}
// over the workgroup's T threads, in every one
template <int T>
__device__ __forceinline__ SamplePart join_all(SamplePart s, int t) {
  __shared__ SamplePart parts[T / 64];
#pragma unroll
  for (int d = 1; d < 64; d *= 2)
    join(s, SamplePart{__shfl_xor(s.top, d, 64), __shfl_xor(s.low, d, 64),
                       (uint32_t)__shfl_xor((int)s.bad, d, 64)});
  if ((t & 63) == 0) parts[t >> 6] = s;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) join(s, parts[w]);
  return s;
}
// of a thread's logits
template <class P>
__device__ __forceinline__ SamplePart survey(const P& part) {
  SamplePart s{-__builtin_inff(), __builtin_inff(), 0};
  bool nan = false;
  part.logits([&](float z, int) {
    nan |= z != z;
    z = __builtin_canonicalizef(z);  // once, not for each of the two
    s.top = fmaxf(s.top, z);
    s.low = fminf(s.low, z == -__builtin_inff() ? __builtin_inff() : z);
  });
  s.bad = nan || s.top == __builtin_inff();
  return s;
}

__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t m, const SamplePart& s) {
  const float temperature = a.temperature ? a.temperature[m] : 1.0f;
  Row r;
  r.l = limits_of(a, m);
  r.top = s.top;
  // (a row without a finite logit has no lowest one)
  r.bad = s.bad || s.low > FLT_MAX || !(temperature < __builtin_inff());
  r.greedy = temperature <= 0.0f;
  r.rate = 1.4426950408889634 / (double)temperature;
  r.floor = fmaxf((float)((double)s.top - (double)(a.bits + 1) / r.rate), -FLT_MAX);
  r.least = -FLT_MAX;
  if (r.l.y > -(double)(a.bits + 1)) {
    // the lowest f32 whose weight is min_p or more: a step or two from the rounded one
    float z = fmaxf((float)((double)s.top + r.l.y / r.rate), -FLT_MAX);
    for (int i = 0; i < 4 && log2_weight(r, z) < r.l.y; ++i) z = nextafterf(z, FLT_MAX);
    for (int i = 0; i < 4 && z > -FLT_MAX; ++i) {
      const float below = nextafterf(z, -FLT_MAX);
      if (log2_weight(r, below) < r.l.y) break;
      z = below;
    }
    r.least = z;
  }
  // without a top-p nothing below min_p's limit enters a sum that decides
  if (r.l.p >= 1.0) r.floor = fmaxf(r.floor, r.least);
  const float range = fminf(r.top - fmaxf(s.low, r.floor), FLT_MAX);
  r.scale = range > 0.0f ? kBins / range : 0.0f;
  // a range so small that the quotient is infinite: one bin
  if (r.scale > FLT_MAX) r.scale = 0.0f;
  return r;
}

// 2^(j / 32), j < 32, in LDS: what weight_of multiplies by.  The caller synchronizes.
constexpr int kRoots = 32;
__device__ __forceinline__ void set_roots(double* roots, int t) {
  if (t < kRoots) roots[t] = exp2((double)t / kRoots);
}
// 2^(x / 32) for x in [-32000, 0] in units of 2^-bits: x = n + f with f in [-1/2, 1/2],
// 2^(n / 32) from the roots, and 2^(f / 32) by its series, with c = ln 2 / 32 to
// (c / 2)^6 / 6! < 10^-14.  (The series of 2^f alone, to f^11, cost twice as much.)  Sums
// with powers of two stand for conversions, which take four times an addition's time.
__device__ __forceinline__ double weight_of(double x, const double* roots, int bits) {
  constexpr double kWhole = 6755399441055744.0;  // 1.5 2^52: n in the sum's low bits
  const double shifted = x + kWhole, f = x - (shifted - kWhole);
  const int i = (int)__builtin_bit_cast(u64, shifted);
  constexpr double c = 0.6931471805599453 / kRoots;
  double p = c * c * c * c * c / 120.0;
  p = fma(p, f, c * c * c * c / 24.0);
  p = fma(p, f, c * c * c / 6.0);
  p = fma(p, f, c * c / 2.0);
  p = fma(p, f, c);
  const u64 power = (u64)(uint32_t)((i >> 5) + bits) << 52;  // added to the exponent
  const double root =
      __builtin_bit_cast(double, __builtin_bit_cast(u64, roots[i & (kRoots - 1)]) + power);
  return fma(p * f, root, root);
}
// as an integer, for a weight of at most 2^50: the low bits of its sum with 2^52
__device__ __forceinline__ u64 rounded(double weight) {
  return __builtin_bit_cast(u64, weight + 4503599627370496.0) & 0xfffffffffffffull;
}
// that of a token from the floor on
__device__ __forceinline__ u64 weight_of(const Row& r, float z, const double* roots, int bits) {
  return rounded(weight_of(((double)z - (double)r.top) * (r.rate * kRoots), roots, bits));
}
// that of any token, not rounded, nothing that counts where z is -inf
__device__ __forceinline__ double exact_weight(const Row& r, float z, const double* roots, int bits) {
  return weight_of(fmax(((double)z - (double)r.top) * (r.rate * kRoots), -32000.0), roots, bits);
}

// ---- launch 1: the largest logit of a part of a row, the lowest finite one, and whether
// the row cannot be drawn from; and its share of what the next launches add to
template <int TYPE>
__global__ __launch_bounds__(kThreads) void top_kernel(SampleArgs a) {
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Part<TYPE> part = part_of<TYPE>(a, m, t);
  for (int b = blockIdx.x * kThreads + t; b < kBins; b += gridDim.x * kThreads) {
    a.count[m * kBins + b] = 0;
    a.weight[m * kBins + b] = 0;
  }
  if (blockIdx.x == 0 && t == 0) a.listed[m] = 0, a.first[m] = 0xffffffffu;
  const SamplePart s = join_all<kThreads>(survey(part), t);
  if (t == 0) a.part[m * a.chunks + blockIdx.x] = s;
}

// a thread's share of the histograms, in LDS
template <class P>
__device__ __forceinline__ void count_tokens(const P& part, const Row& r, uint32_t* count) {
  part.logits([&](float z, int) {
    if (z >= r.floor) atomicAdd(&count[bin_of(r, z)], 1u);
  });
}
// and the thread's exact sum of a row's weights where the logarithm of a share needs it
template <class P>
__device__ __forceinline__ double sum_weights(const P& part, const Row& r, u64* weight,
                                              const double* roots, int bits) {
  double sum = 0.0;
  if (r.exact()) {
    const float from = r.l.y < -100.0 ? -__builtin_inff() : r.least;
    part.logits([&](float z, int) {
      const double w = exact_weight(r, z, roots, bits);
      sum += z >= from ? w : 0.0;
      if (z >= r.floor) atomicAdd(&weight[bin_of(r, z)], rounded(w));
    });
  } else {
    part.logits([&](float z, int) {
      if (z >= r.floor) atomicAdd(&weight[bin_of(r, z)], weight_of(r, z, roots, bits));
    });
  }
  return sum;
}

// ---- what the histograms say

// inclusive sums over the workgroup's threads, in their order
template <int T>
__device__ __forceinline__ void scan(uint32_t& c, u64& w, int t) {
  __shared__ uint32_t cs[T / 64];
  __shared__ u64 ws[T / 64];
  const int lane = t & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t oc = (uint32_t)__shfl_up((int)c, d, 64);
    const u64 ow = (u64)__shfl_up((long long)w, d, 64);
    if (lane >= d) c += oc, w += ow;
  }
  __syncthreads();  // the last use of cs and ws has ended
  if (lane == 63) cs[t >> 6] = c, ws[t >> 6] = w;
  __syncthreads();
  for (int i = 0; i < t >> 6; ++i) c += cs[i], w += ws[i];
}

// Weights of a row before each bin, with the whole row's behind the last
struct Sums {
  u64 weight[kBins + 1];
};

// where a sum's bounds [lo, hi] put the place that it decides
struct Bounds {
  u64 lo, hi;
};

// The bin that holds the k-th token, and the tokens ahead of the bin; where there are fewer
// than k the last bin, and kFewer.
constexpr uint32_t kFewer = 0xffffffffu;
template <int T>
__device__ __forceinline__ int kth_bin(const uint32_t* count, int t, uint32_t k, uint32_t& ahead) {
  constexpr int B = kBins / T;
  __shared__ int at;
  __shared__ uint32_t before;
  uint32_t c[B], sum = 0;
  u64 none = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) sum += c[i] = count[B * t + i];
  uint32_t past = sum;
  if (t == 0) at = kBins - 1, before = kFewer;
  scan<T>(past, none, t);  // synchronizes
  past -= sum;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    if (past < k && past + c[i] >= k) at = B * t + i, before = past;
    past += c[i];
  }
  __syncthreads();
  ahead = before;
  return at;
}

// The bins whose tokens decide a row by sums: a range for each place.
struct Needed {
  int lo[4], hi[4];
  int kth;         // with a k: its bin
  uint32_t ahead;  // and the tokens ahead of that bin
};

// Sums the row's histogram of weights (and with a k reads that of tokens), and says which
// bins decide its token.
template <int T>
__device__ __forceinline__ Needed plan(const Row& r, const uint32_t* count, const u64* weight,
                                       int bits, int t, Sums& s) {
  constexpr int B = kBins / T;
  __shared__ int at[4];
  const Limits& l = r.l;
  u64 w[B], ws = 0;
  uint32_t none = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) ws += w[i] = weight[B * t + i];
  u64 wi = ws;
  scan<T>(none, wi, t);
  wi -= ws;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    s.weight[B * t + i] = wi;
    wi += w[i];
  }
  if (t == T - 1) s.weight[kBins] = wi;
  if (t < 4) at[t] = 0;
  Needed n;
#pragma unroll
  for (int i = 0; i < 4; ++i) n.lo[i] = 1, n.hi[i] = 0;  // none
  n.kth = 0;
  if (l.k > 0) n.kth = kth_bin<T>(count, t, (uint32_t)l.k, n.ahead);
  __syncthreads();

  const u64 all = s.weight[kBins];
  Bounds k{all, all};
  if (l.k > 0) {
    n.lo[0] = n.hi[0] = n.kth;
    k = Bounds{s.weight[n.kth], s.weight[n.kth + 1]};
  }
  Bounds p = k;
  if (r.by_p()) {
    const double lo = l.p * (double)k.lo, hi = l.p * (double)k.hi;
    for (int b = B * t; b < B * t + B; ++b) {
      const double before = (double)s.weight[b], past = (double)s.weight[b + 1];
      if (before < lo && past >= lo) at[0] = b;  // (none where lo is 0: bin 0)
      if (before < hi && past >= hi) at[1] = b;
    }
    __syncthreads();
    n.lo[1] = at[0], n.hi[1] = at[1];
    p = Bounds{s.weight[n.lo[1]], min(s.weight[n.hi[1] + 1], k.hi)};
  } else if (l.p <= 0.0) {
    p.lo = p.hi = 1ull << bits;  // the first token alone
  }
  Bounds q = p;
  if (r.by_q()) {
    n.lo[2] = n.hi[2] = bin_of(r, r.least);
    q = Bounds{min(p.lo, s.weight[n.lo[2]]), min(p.hi, s.weight[n.lo[2] + 1])};
  }
  const double lo = l.u * (double)q.lo, hi = l.u * (double)q.hi;
  for (int b = B * t; b < B * t + B; ++b) {
    const double before = (double)s.weight[b], past = (double)s.weight[b + 1];
    if (before <= lo && past > lo) at[2] = b;
    if (before <= hi && past > hi) at[3] = b;
  }
  __syncthreads();
  n.lo[3] = at[2], n.hi[3] = at[3];
  return n;
}

__device__ __forceinline__ Ranges ranges_down_to(int bin) {
  return Ranges{{0.0f, 1.0f, 1.0f, 1.0f}, {past(bin), 0.0f, 0.0f, 0.0f}, true};
}
__device__ __forceinline__ Ranges ranges_of(const Needed& n) {
  Ranges g;
  g.one = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool some = n.lo[i] <= n.hi[i];
    g.lo[i] = some ? (float)n.lo[i] : 1.0f;
    g.hi[i] = some ? past(n.hi[i]) : 0.0f;
  }
  return g;
}

// ---- launch 2: the histograms: of tokens where a k decides, of weights where it is not
// small (both, one after the other, for the few rows of a large k)
template <int TYPE>
__global__ __launch_bounds__(kThreads) void histogram_kernel(SampleArgs a) {
  __shared__ u64 bins[kBins];
  __shared__ double roots[kRoots], sums[kThreads / 64];
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Part<TYPE> part = part_of<TYPE>(a, m, t);
  for (int b = t; b < kBins; b += kThreads) bins[b] = 0;
  set_roots(roots, t);
  SamplePart all{-__builtin_inff(), __builtin_inff(), 0};
  for (int c = t; c < a.chunks; c += kThreads) join(all, a.part[m * a.chunks + c]);
  const Row r = row_of(a, m, join_all<kThreads>(all, t));  // synchronizes
  if (blockIdx.x == 0 && t == 0) rows_of(a)[m].row = r;
  if (r.bad || r.greedy) return;  // all of the row's workgroups
  if (r.l.k > 0) {
    uint32_t* count = reinterpret_cast<uint32_t*>(bins);
    count_tokens(part, r, count);
    __syncthreads();
    for (int b = t; b < kBins; b += kThreads)
      if (count[b]) atomicAdd(a.count + m * kBins + b, count[b]);
    if (r.listed()) return;
    __syncthreads();
    for (int b = t; b < kBins / 2; b += kThreads) bins[b] = 0;
    __syncthreads();
  }
  double sum[1] = {sum_weights(part, r, bins, roots, a.bits)};
  if (r.exact()) {
    sum_all<kThreads>(sum, sums, t);
    if (t == 0) a.sum[m * a.chunks + blockIdx.x] = sum[0];
  }
  __syncthreads();
  for (int b = t; b < kBins; b += kThreads)
    if (bins[b]) atomicAdd(a.weight + m * kBins + b, bins[b]);
}

// What is gathered of a row that is neither greedy nor bad
template <int T>
__device__ __forceinline__ Ranges ranges_of(const SampleArgs& a, const Row& r, int64_t m, int t,
                                            Sums& s) {
  const uint32_t* count = a.count + m * kBins;
  if (!r.listed()) return ranges_of(plan<T>(r, count, a.weight + m * kBins, a.bits, t, s));
  uint32_t ahead;
  return ranges_down_to(kth_bin<T>(count, t, (uint32_t)r.l.k, ahead));
}

// That in a launch of its own, for many rows (kPlanned): each workgroup of the gathering would
// read the row's histogram again (rows of 151936 in f32 with a top-p, us, worked out there / by
// a launch: one row 24.0 / 24.5, 16 rows 65 / 60, 32 rows 60 / 54, 128 rows 116 / 101).
__global__ __launch_bounds__(kDraw) void plan_kernel(SampleArgs a) {
  __shared__ Sums s;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Row r = rows_of(a)[m].row;
  if (r.bad || r.greedy) return;
  const Ranges g = ranges_of<kDraw>(a, r, m, t, s);
  if (t == 0) rows_of(a)[m].ranges = g;
}

// ---- launch 3: the tokens of those bins
// take(v, index of v[0], which of them) for a thread's pieces with tokens in the ranges
template <class P, class Take>
__device__ __forceinline__ void select(const P& part, const Row& r, const Ranges& g, Take take) {
  constexpr int V = P::V;
  // what lies below the floor has places from about kBins on, or where all else is equal the
  // same one as that
  const float ends = g.hi[0] + g.hi[1] + g.hi[2] + g.hi[3];
  const bool apart = ends == ends && r.scale > 0.0f;
  if (g.one && apart) {
    const float far = g.hi[0];
    part.pieces([&](const float(&v)[V], int n) {
      uint32_t mask = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) mask |= place_of(r, v[e]) < far ? 1u << e : 0u;
      if (mask) take(v, n, mask);
    });
    return;
  }
  part.pieces([&](const float(&v)[V], int n) {
    float x[V];
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = place_of(r, v[e]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(g.lo[i] >= g.hi[i])) {  // the same in all lanes
#pragma unroll
        for (int e = 0; e < V; ++e) mask |= x[e] >= g.lo[i] && !(x[e] >= g.hi[i]) ? 1u << e : 0u;
      }
    if (!apart) {
#pragma unroll
      for (int e = 0; e < V; ++e) mask &= v[e] >= r.floor ? ~0u : ~(1u << e);
    }
    if (mask) take(v, n, mask);
  });
}

// The workgroup's are listed in LDS first, a place there for all of a thread's piece at a
// time, and then behind the row's others: one atomic in memory for all of them (with one for
// each token 128 rows took 38 us).  What does not fit there goes to the row's list at once.
constexpr int kMine = kList / 2;
template <int TYPE, bool PLANNED>
__global__ __launch_bounds__(kThreads) void gather_kernel(SampleArgs a) {
  constexpr int V = kValues<TYPE>;
  __shared__ union {
    Sums sums;  // not PLANNED: until the places are known
    u64 mine[kMine];
  } lds;
  __shared__ uint32_t taken, base;
  u64* mine = lds.mine;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Part<TYPE> part = part_of<TYPE>(a, m, t);
  const Row r = rows_of(a)[m].row;
  if (r.bad) return;
  if (t == 0) taken = 0;
  __syncthreads();
  if (r.greedy) {
    uint32_t first = 0xffffffffu;
    part.logits([&](float z, int n) { first = z == r.top ? min(first, (uint32_t)n) : first; });
    if (first != 0xffffffffu) atomicMin(a.first + m, first);
    return;
  }
  Ranges ranges;
  if constexpr (PLANNED) {
    ranges = rows_of(a)[m].ranges;
  } else {
    ranges = ranges_of<kThreads>(a, r, m, t, lds.sums);
    __syncthreads();  // the sums' place is the list's
  }
  select(part, r, ranges, [&](const float(&v)[V], int n, uint32_t mask) {
    uint32_t at = atomicAdd(&taken, (uint32_t)__popc(mask));
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (mask >> e & 1) {
        if (at < kMine) {
          mine[at] = entry_of(v[e], n + e);
        } else {
          const uint32_t i = atomicAdd(a.listed + m, 1u);
          if (i < kList) a.list[m * kList + i] = entry_of(v[e], n + e);
        }
        ++at;
      }
  });
  __syncthreads();
  const uint32_t count = min(taken, (uint32_t)kMine);
  if (t == 0) base = count ? atomicAdd(a.listed + m, count) : 0;
  __syncthreads();
  for (uint32_t i = t; i < count; i += kThreads)
    if (base + i < kList) a.list[m * kList + base + i] = mine[i];
}

// ---- launch 4: the draw

// the first place whose sum is at least (past: more than) `to`, n places of equal weight w
// each behind `base`: 1 .. n
__device__ __forceinline__ uint32_t place_among(u64 base, u64 w, uint32_t n, double to, bool past) {
  uint32_t lo = 1, hi = n;
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const double sum = (double)(base + mid * w);
    if (past ? sum > to : sum >= to)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// A place in the order found by the bits of the logits, eight at a time, over the whole
// row: where so many tokens share the bins that they cannot be sorted.
struct Found {
  uint32_t key, before, ties;  // its logit, the tokens ahead of all that share it, how many do
  u64 sum, weight;             // their weights' sum, and the weight of each that shares it
};
enum Search { kByCount, kBySum, kPastSum };

template <int TYPE>
__device__ __forceinline__ Found search(const SampleArgs& a, const Row& r, const double* roots,
                                        int64_t m, int t, Search how, uint32_t k, double to) {
  __shared__ uint32_t count[256], digit, found_before, found_ties;
  __shared__ u64 weight[256], found_sum, found_weight;
  uint32_t prefix = 0, before = 0;
  u64 sum = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (t < 256) count[t] = 0, weight[t] = 0;
    __syncthreads();
    for_row<TYPE, kDraw>(a, m, t, [&](float z, int) {
      const uint32_t key = key_of(z);
      if (!(z >= r.floor) || (shift < 24 && key >> (shift + 8) != prefix)) return;
      const int b = 255 - (key >> shift & 255);  // the largest first
      atomicAdd(&count[b], 1u);
      atomicAdd(&weight[b], weight_of(r, z, roots, a.bits));
    });
    __syncthreads();
    const uint32_t mine = t < 256 ? count[t] : 0;
    const u64 mine_w = t < 256 ? weight[t] : 0;
    uint32_t c = mine;
    u64 w = mine_w;
    scan<kDraw>(c, w, t);
    c += before, w += sum;
    const double ahead = (double)(w - mine_w), past = (double)w;
    const bool here = how == kByCount ? c - mine < k && c >= k
                      : how == kBySum ? ahead < to && past >= to
                                      : ahead <= to && past > to;
    if (here && mine) {
      digit = 255 - t;
      found_before = c - mine, found_ties = mine;
      found_sum = w - mine_w, found_weight = mine_w;
    }
    __syncthreads();
    prefix = prefix << 8 | digit;
    before = found_before, sum = found_sum;
  }
  // (the barriers above are ahead of the next search's writes of what is read here)
  const Found f{prefix, before, found_ties, sum, found_weight / found_ties};
  __syncthreads();
  return f;
}

// the index of the place-th (from 1) of the row's logits that have this key
template <int TYPE>
__device__ __forceinline__ int64_t index_of(const SampleArgs& a, int64_t m, int t, uint32_t key,
                                            uint32_t place) {
  __shared__ int result;
  uint32_t seen = 0;
  for (int64_t n0 = 0; n0 < a.N; n0 += kDraw) {
    const int64_t n = n0 + t;
    const bool is = n < a.N && key_of(load_as_f32(a.Z, m * a.ldz + n, TYPE)) == key;
    uint32_t c = is;
    u64 w = 0;
    scan<kDraw>(c, w, t);
    if (is && seen + c == place) result = (int)n;
    seen += __syncthreads_count(is);
    if (seen >= place) break;  // all threads
  }
  return result;
}

// the draw's LDS
struct Draw {
  Sums s;
  uint32_t start[kBins];  // a needed bin's first place in the list
  u64 list[kList], ahead[kList + 1];
  double roots[kRoots], sums[kDraw / 64];
  u64 found, below;
  uint32_t tokens;
  int which;
};

// list[0 .. size) in descending order, size a power of two from 64 on: a bitonic sort, its
// steps across less than 64 places in the lanes of a wave
__device__ __forceinline__ void sort(u64* list, int size, int t) {
  const int lane = t & 63, wave = t >> 6;
  // the steps j = from, from / 2 .. 1 of level k on the wave's 64 places from `at` on
  auto within = [&](u64 v, int at, int k, int from) {
    const bool down = ((at + lane) & k) == 0;
    for (int j = from; j > 0; j /= 2) {
      const u64 o = (u64)__shfl_xor((long long)v, j, 64);
      const bool first = (lane & j) == 0;
      v = (first == down) == (v > o) ? v : o;  // (equal entries are zeros)
    }
    return v;
  };
  for (int at = 64 * wave; at < size; at += kDraw) {
    u64 v = list[at + lane];
    for (int k = 2; k <= 64; k *= 2) v = within(v, at, k, k / 2);
    list[at + lane] = v;
  }
  for (int k = 128; k <= size; k *= 2) {
    for (int j = k / 2; j >= 64; j /= 2) {
      __syncthreads();
      for (int i = t; i < size / 2; i += kDraw) {
        const int lo = 2 * (i - (i & (j - 1))) + (i & (j - 1)), hi = lo + j;
        const u64 x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) list[lo] = y, list[hi] = x;
      }
    }
    __syncthreads();
    for (int at = 64 * wave; at < size; at += kDraw)
      list[at + lane] = within(list[at + lane], at, k, 32);
  }
  __syncthreads();
}

// What a sum of weights has beyond the first token's, in units of that
__device__ __forceinline__ double beyond_first(u64 whole, int bits) {
  return __builtin_ldexp((double)(whole - (1ull << bits)), -bits);
}

struct Drawn {
  u64 entry;      // the token's
  double others;  // beyond_first of what it was drawn from
};

// The token from the sorted list of `count` tokens, at most E of each thread.
template <int E>
__device__ __forceinline__ Drawn resolve(const SampleArgs& a, const Row& r, const Needed& need,
                                         Draw& d, int count, int t) {
  const Limits& l = r.l;
  const bool listed = r.listed();
  if (t == 0) d.below = 0, d.which = 0;
  // weights of places E t .. E t + E - 1 of the list, and the sums ahead of them
  u64 w[E], sum = 0;
  int bin[E];
  float z[E];
  int previous = -1;
  if (!listed && t > 0 && E * t < count)
    previous = bin_of(r, value_of((uint32_t)(d.list[E * t - 1] >> 32)));
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = E * t + e;
    w[e] = 0, bin[e] = 0, z[e] = 0.0f;
    if (i < count) {
      z[e] = value_of((uint32_t)(d.list[i] >> 32));
      w[e] = weight_of(r, z[e], d.roots, a.bits);
      bin[e] = bin_of(r, z[e]);
      if (!listed && bin[e] != previous) d.start[bin[e]] = i;
      previous = bin[e];
    }
    sum += w[e];
  }
  uint32_t none = 0;
  u64 total = sum;
  scan<kDraw>(none, total, t);
  u64 before = total - sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    d.ahead[E * t + e] = before;
    before += w[e];
  }
  if (t == kDraw - 1) d.ahead[E * kDraw] = before;
  __syncthreads();
  // the sum of all weights of the row ahead of the thread's places (by sums: its bin's, and the
  // list's ahead of it in the bin)
  u64 from[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = E * t + e;
    from[e] = 0;
    if (i < count)
      from[e] = listed ? d.ahead[i]
                       : d.s.weight[bin[e]] + (d.ahead[i] - d.ahead[d.start[bin[e]]]);
  }

  u64 whole = listed ? d.ahead[min(l.k, count)] : d.s.weight[kBins];
  if (!listed && l.k > 0 && need.ahead != kFewer) {
    const uint32_t first = d.start[need.kth];
    whole = d.s.weight[need.kth] + (d.ahead[first + (l.k - need.ahead)] - d.ahead[first]);
  }
  if (r.by_p()) {
    const double to = l.p * (double)whole;
    if (t == 0) d.found = whole;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (E * t + e < count && (double)from[e] < to && (double)(from[e] + w[e]) >= to)
        d.found = min(whole, from[e] + w[e]);
    __syncthreads();
    whole = d.found;
  } else if (l.p <= 0.0) {
    whole = 1ull << a.bits;
  }
  if (r.by_q()) {
    // (all of a list down to the k-th; else those of the limit's bin and all ahead of it)
    u64 mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (E * t + e < count && z[e] >= r.least && (listed || bin[e] == need.lo[2])) mine += w[e];
    if (mine) atomicAdd(&d.below, mine);
    __syncthreads();
    whole = min(whole, listed ? d.below : d.s.weight[need.lo[2]] + d.below);
  }
  const double to = l.u * (double)whole;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (E * t + e < count && (double)from[e] <= to && (double)(from[e] + w[e]) > to)
      d.which = E * t + e;
  __syncthreads();
  double others[1] = {0.0};
  if (listed) {
    // those of the list, exactly
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (E * t + e > 0 && E * t + e < count && from[e] + w[e] <= whole)
        others[0] += exact_weight(r, z[e], d.roots, 0);
    sum_all<kDraw>(others, d.sums, t);
  } else {
    others[0] = beyond_first(whole, a.bits);
  }
  return Drawn{d.list[d.which], others[0]};
}

// The token of a row that is neither greedy nor bad, from its list of `count` tokens in
// d.list (more than kList: not all are there); the roots are set.  `sum`: an exact() row's.
template <int TYPE>
__device__ __forceinline__ void draw(const SampleArgs& a, const Row& r, const Needed& need,
                                     int64_t m, int t, Draw& d, int count, double sum) {
  const Limits& l = r.l;
  auto finish = [&](int64_t token, float z, double others) {
    if (r.exact()) others = __builtin_ldexp(sum, -a.bits) - 1.0;
    a.token[m] = token;
    if (a.logprob) a.logprob[m] = (float)(0.6931471805599453 * log2_weight(r, z) - log1p(others));
  };
  if (count > kList) {  // all of the workgroup
    // how many tokens there are, and the sums of all and of those from min_p on
    if (t == 0) d.found = 0, d.below = 0, d.tokens = 0;
    __syncthreads();
    u64 mine = 0, kept = 0;
    uint32_t some = 0;
    for_row<TYPE, kDraw>(a, m, t, [&](float z, int) {
      if (!(z >= r.floor)) return;
      const u64 w = weight_of(r, z, d.roots, a.bits);
      some += 1;
      mine += w;
      kept += z >= r.least ? w : 0;
    });
    atomicAdd(&d.tokens, some);
    atomicAdd(&d.found, mine);
    atomicAdd(&d.below, kept);
    __syncthreads();
    u64 whole = d.found;
    if (l.k > 0 && (uint32_t)l.k < d.tokens) {
      const Found f = search<TYPE>(a, r, d.roots, m, t, kByCount, (uint32_t)l.k, 0.0);
      whole = f.sum + (l.k - f.before) * f.weight;
    }
    if (r.by_p()) {
      const double to = l.p * (double)whole;
      const Found f = search<TYPE>(a, r, d.roots, m, t, kBySum, 0, to);
      whole = min(whole, f.sum + place_among(f.sum, f.weight, f.ties, to, false) * f.weight);
    } else if (l.p <= 0.0) {
      whole = 1ull << a.bits;
    }
    if (r.by_q()) whole = min(whole, d.below);
    const double to = l.u * (double)whole;
    const Found f = search<TYPE>(a, r, d.roots, m, t, kPastSum, 0, to);
    const uint32_t place = place_among(f.sum, f.weight, f.ties, to, true);
    const int64_t token = index_of<TYPE>(a, m, t, f.key, place);
    if (t == 0) finish(token, value_of(f.key), beyond_first(whole, a.bits));
    return;
  }


  // sorted in descending order, zeros (no token's entry) behind them
  int size = 64;
  while (size < count) size *= 2;
  for (int i = count + t; i < size; i += kDraw) d.list[i] = 0;
  __syncthreads();
  sort(d.list, size, t);
  const Drawn it = count <= kDraw ? resolve<1>(a, r, need, d, count, t)
                                  : resolve<kList / kDraw>(a, r, need, d, count, t);
  if (t == 0) finish((uint32_t)~(uint32_t)it.entry, value_of((uint32_t)(it.entry >> 32)), it.others);
}

// a greedy row's token, or none
__device__ __forceinline__ void draw_first(const SampleArgs& a, const Row& r, int64_t m,
                                           uint32_t first) {
  a.token[m] = r.bad ? -1 : (int64_t)first;
  if (a.logprob) a.logprob[m] = r.bad ? __builtin_nanf("") : 0.0f;
}

template <int TYPE>
__global__ __launch_bounds__(kDraw) void draw_kernel(SampleArgs a) {
  __shared__ Draw d;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Row r = rows_of(a)[m].row;
  if (r.bad || r.greedy) {
    if (t == 0) draw_first(a, r, m, a.first[m]);
    return;
  }
  const int count = (int)min(a.listed[m], (uint32_t)kList + 1);
  set_roots(d.roots, t);
  for (int i = t; i < count && count <= kList; i += kDraw) d.list[i] = a.list[m * kList + i];
  Needed need;
  if (!r.listed())
    need = plan<kDraw>(r, a.count + m * kBins, a.weight + m * kBins, a.bits, t, d.s);
  double sum[1] = {0.0};
  if (r.exact())
    for (int c = t; c < a.chunks; c += kDraw) sum[0] += a.sum[m * a.chunks + c];
  sum_all<kDraw>(sum, d.sums, t);  // synchronizes
  draw<TYPE>(a, r, need, m, t, d, count, sum[0]);
}

// ---- all of it in one launch, for rows that a workgroup holds in registers
constexpr int kWhole = 16;  // 16-byte pieces a thread
template <int TYPE>
__global__ __launch_bounds__(kDraw) void whole_kernel(SampleArgs a) {
  constexpr int V = kValues<TYPE>;
  __shared__ Draw d;
  __shared__ uint32_t taken, first;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Part<TYPE, kDraw, kWhole> part(a, m, 0, a.N, t);
  // the histograms, in places that are used after them
  uint32_t* count = d.start;
  u64* weight = d.ahead;
  static_assert(kBins <= kList, "a bin a place");
  for (int b = t; b < kBins; b += kDraw) count[b] = 0, weight[b] = 0;
  if (t == 0) taken = 0, first = 0xffffffffu;
  set_roots(d.roots, t);
  const Row r = row_of(a, m, join_all<kDraw>(survey(part), t));  // synchronizes
  if (r.bad || r.greedy) {
    uint32_t mine = 0xffffffffu;
    part.logits([&](float z, int n) { mine = z == r.top ? min(mine, (uint32_t)n) : mine; });
    if (mine != 0xffffffffu) atomicMin(&first, mine);
    __syncthreads();
    if (t == 0) draw_first(a, r, m, first);
    return;
  }
  Needed need;
  Ranges ranges;
  if (r.l.k > 0) count_tokens(part, r, count);
  double sum[1] = {0.0};
  if (!r.listed()) sum[0] = sum_weights(part, r, weight, d.roots, a.bits);
  sum_all<kDraw>(sum, d.sums, t);  // synchronizes
  if (r.listed()) {
    uint32_t ahead;
    ranges = ranges_down_to(kth_bin<kDraw>(count, t, (uint32_t)r.l.k, ahead));
  } else {
    need = plan<kDraw>(r, count, weight, a.bits, t, d.s);
    ranges = ranges_of(need);
  }
  select(part, r, ranges, [&](const float(&v)[V], int n, uint32_t mask) {
    uint32_t at = atomicAdd(&taken, (uint32_t)__popc(mask));
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (mask >> e & 1) {
        if (at < kList) d.list[at] = entry_of(v[e], n + e);
        ++at;
      }
  });
  __syncthreads();
  draw<TYPE>(a, r, need, m, t, d, (int)min(taken, (uint32_t)kList + 1), sum[0]);
}

// Whether a row goes through one launch: as long as it fits, and where there are few rows
// while one workgroup is not slower than the parts of a row (us, one launch / four, with a
// top-p alone and replayed from a graph: one row of 16000 in f32 17 / 21, of 32000 26 / 21; 16
// rows of 32000 26 / 26, of 40000 in bf16 33 / 27; 128 rows of 32000 28 / 44, of 65536 in bf16
// 51 / 52; 512 of those 102 / 119)
bool is_whole(int type, int64_t M, int64_t N) {
  const int64_t fits = (type == GEMMQ_F32 ? 4 : 8) * kWhole * kDraw;
  return N <= fits && (N <= 16384 || (M >= 16 && N <= 32768) || M >= 128);
}

// rows of a set of launches: bounds the workspace, and the grid
constexpr int64_t kRows = 1024, kWholeRows = 32768;
constexpr int64_t kPlanned = 32;  // rows from which the plan has its own launch

struct Layout {
  int64_t rows, chunks, chunk;
  size_t weight, list, sum, rows_at, part, count, listed, first, bytes;
};

// Parts of a row: the largest that leave a launch 1024 workgroups, of two pieces a thread at
// least
Layout layout(int type, int64_t M, int64_t N) {
  Layout l;
  l.rows = M < kRows ? M : kRows;
  const int64_t span = (type == GEMMQ_F32 ? 4 : 8) * kThreads;
  int64_t pieces = kMostOfARow / span;
  while (pieces > 2 && l.rows * ceil_div(N, pieces * span) < 1024) pieces /= 2;
  l.chunk = pieces * span;
  l.chunks = ceil_div(N, l.chunk);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)ceil_div(bytes, 256) * 256;
    return here;
  };
  l.weight = take(8 * l.rows * kBins);
  l.list = take(8 * l.rows * kList);
  l.sum = take(8 * l.rows * l.chunks);
  l.rows_at = take((int64_t)sizeof(RowAndRanges) * l.rows);
  l.part = take((int64_t)sizeof(SamplePart) * l.rows * l.chunks);
  l.count = take(4 * l.rows * kBins);
  l.listed = take(4 * l.rows);
  l.first = take(4 * l.rows);
  l.bytes = at;
  return l;
}

template <int TYPE>
void launch_type(const SampleArgs& a, int rows, bool whole, hipStream_t st) {
  const dim3 grid((uint32_t)a.chunks, (uint32_t)rows), one(1, (uint32_t)rows);
  if (whole) {
    whole_kernel<TYPE><<<one, kDraw, 0, st>>>(a);
    return;
  }
  top_kernel<TYPE><<<grid, kThreads, 0, st>>>(a);
  histogram_kernel<TYPE><<<grid, kThreads, 0, st>>>(a);
  if (rows >= kPlanned) {
    plan_kernel<<<one, kDraw, 0, st>>>(a);
    gather_kernel<TYPE, true><<<grid, kThreads, 0, st>>>(a);
  } else {
    gather_kernel<TYPE, false><<<grid, kThreads, 0, st>>>(a);
  }
  draw_kernel<TYPE><<<one, kDraw, 0, st>>>(a);
}

}  // namespace

size_t sample_workspace(int64_t M, int64_t N) {
  // f32's parts are the smaller ones, and where its rows go through one launch all do
  return is_whole(GEMMQ_F32, M, N) ? 0 : layout(GEMMQ_F32, M, N).bytes;
}

int launch_sample(SampleArgs a, int type, int64_t M, void* ws, hipStream_t st) {
  int log = 0;
  while (((int64_t)1 << log) < a.N) ++log;
  a.bits = 62 - log < 50 ? 62 - log : 50;
  const bool whole = is_whole(type, M, a.N);
  int64_t each = M < kWholeRows ? M : kWholeRows;
  if (!whole) {
    const Layout l = layout(type, M, a.N);
    uint8_t* p = static_cast<uint8_t*>(ws);
    a.weight = reinterpret_cast<u64*>(p + l.weight);
    a.list = reinterpret_cast<u64*>(p + l.list);
    a.sum = reinterpret_cast<double*>(p + l.sum);
    a.rows = p + l.rows_at;
    a.part = reinterpret_cast<SamplePart*>(p + l.part);
    a.count = reinterpret_cast<uint32_t*>(p + l.count);
    a.listed = reinterpret_cast<uint32_t*>(p + l.listed);
    a.first = reinterpret_cast<uint32_t*>(p + l.first);
    a.chunk = (int)l.chunk;
    a.chunks = (int)l.chunks;
    each = l.rows;
  }
  for (int64_t m = 0; m < M; m += each) {
    const int rows = (int)(M - m < each ? M - m : each);
    type == GEMMQ_F32    ? launch_type<GEMMQ_F32>(a, rows, whole, st)
    : type == GEMMQ_BF16 ? launch_type<GEMMQ_BF16>(a, rows, whole, st)
                         : launch_type<GEMMQ_F16>(a, rows, whole, st);
    a.Z = static_cast<const uint8_t*>(a.Z) + each * a.ldz * type_bytes(type);
    if (a.temperature) a.temperature += each;
    if (a.top_k) a.top_k += each;
    if (a.top_p) a.top_p += each;
    if (a.min_p) a.min_p += each;
    a.u += each;
    a.token += each;
    if (a.logprob) a.logprob += each;
  }
  return 0;
}

}  // namespace i8
}  // namespace gemmq
