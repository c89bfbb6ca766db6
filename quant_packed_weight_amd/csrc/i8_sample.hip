// i8_sample.hip -- one token a row from its logits (gemmq_sample): temperature, top-k,
// top-p, min-p and a given random number, without sorting the vocabulary.
//
// The tokens stand in descending order of their logits (equal ones by index), and every
// limit keeps a prefix of that order, so all that is asked for are places in it: where the
// count reaches k, where the sum of the weights reaches p of what that leaves, where the
// weights fall below min_p, and where the sum passes u of what all of them leave.  A
// histogram over the distance from the largest logit (a function of the logit that never
// rises, so its bins are in that order) gives each place's bin; only those bins' tokens
// are gathered and sorted.  Bounds of the sums that a limit leaves give a range of
// bins where the one before it has not been resolved within its bin yet.
//
// Four launches: the rows' maxima; the histograms; the gathering; the draw.  A row is
// spread over as many workgroups as fill the chip, but for the draw.
//
// Weights are integers, e = exp((z - max) / t) in units of 2^-s: their sums are exact, so
// atomics may add them in any order.  e is computed in f64, to 10^-14: with f32's 10^-7 one
// row in a few hundred of a flat distribution would draw the neighbour of the token that
// the definition draws.
#include "i8_block.h"
#include "i8_common.h"

namespace gemmq {
namespace i8 {
namespace {

typedef unsigned long long u64;

constexpr int kBins = 1024;   // of a row's histogram
constexpr int kList = 4096;   // tokens that are sorted; a row whose bins hold more is searched
                              // by its logits' bits instead (as where all logits are equal)
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

__device__ __forceinline__ u64 shuffle_xor(u64 v, int d) {
  return (u64)__shfl_xor((long long)v, d, 64);
}

// goes through logits [begin, end) of row m in 16-byte pieces; each(z, index)
template <int TYPE, int T, class Each>
__device__ __forceinline__ void for_logits(const SampleArgs& a, int64_t m, int begin, int end, int t,
                                           Each each) {
  constexpr int V = kValues<TYPE>;
  for (int n = begin + V * t; n < end; n += V * T) {
    float v[V];
    load_values<TYPE, V>(a.Z, m * a.ldz + n, end - n, a.wide, v);
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (n + e < end) each(v[e], n + e);
  }
}

// What a row's launches after the first know of it, from the parts' maxima and the row's
// settings (in every thread)
struct Row {
  double top;     // the largest logit
  double rate;    // log2 e / temperature
  double scale;   // bins per unit of distance
  int64_t token;  // of the largest logit
  bool bad, greedy;
};

template <int T>
__device__ __forceinline__ Row row_of(const SampleArgs& a, int64_t m, int t) {
  __shared__ u64 tops[T / 64];
  __shared__ uint32_t lows[T / 64], bads[T / 64];
  u64 top = 0;
  uint32_t low = 0xffffffffu, bad = 0;
  for (int c = t; c < a.chunks; c += T) {
    const SamplePart p = a.part[m * a.chunks + c];
    top = max(top, p.top);
    low = min(low, p.low);
    bad |= p.bad;
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    top = max(top, shuffle_xor(top, d));
    low = min(low, (uint32_t)__shfl_xor((int)low, d, 64));
    bad |= (uint32_t)__shfl_xor((int)bad, d, 64);
  }
  if ((t & 63) == 0) tops[t >> 6] = top, lows[t >> 6] = low, bads[t >> 6] = bad;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 64; ++w) {
    top = max(top, tops[w]);
    low = min(low, lows[w]);
    bad |= bads[w];
  }
  const float temperature = a.temperature ? a.temperature[m] : 1.0f;
  Row r;
  const float z = value_of((uint32_t)(top >> 32));
  r.token = (uint32_t)~(uint32_t)top;
  r.top = z;
  // (a row without a finite logit has no lowest one)
  r.bad = bad || low == 0xffffffffu || !(temperature < __builtin_inff());
  r.greedy = temperature <= 0.0f;
  r.rate = 1.4426950408889634 / (double)temperature;
  // from the largest logit to the lowest, or to where the weights are zero
  const double range =
      fmin(r.top - (double)value_of(low), (double)(a.bits + 1) / r.rate);
  r.scale = range > 0.0 ? kBins / range : 0.0;
  return r;
}

// log2 of a token's weight relative to the largest, <= 0; below -(bits + 1) the weight is
// zero and the token counts nowhere
__device__ __forceinline__ double log2_weight(const Row& r, double distance) {
  return -distance * r.rate;
}
__device__ __forceinline__ int bin_of(const Row& r, double distance) {
  return (int)fmin(distance * r.scale, (double)(kBins - 1));
}

// 2^y for y in [-(bits + 1), 0] in units of 2^-bits, rounded; 2^r by its series, r in
// [-1/2, 1/2], to r^12 (ln 2)^12 / 12! < 10^-14
__device__ __forceinline__ u64 weight_of(double y, int bits) {
  const double n = rint(y), r = (y - n) * 0.6931471805599453;
  double p = 1.0 / 39916800.0;
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  // at most 2^50: the sum with 2^52 holds the integer in its low bits
  const double s = __builtin_ldexp(p, (int)n + bits) + 4503599627370496.0;
  return __builtin_bit_cast(u64, s) & 0xfffffffffffffull;
}

// ---- launch 1: the largest logit and its place, the lowest finite one, and whether the
// row cannot be drawn from, of a part of a row; and its share of what the next launches add to
template <int TYPE>
__global__ __launch_bounds__(kThreads) void top_kernel(SampleArgs a) {
  __shared__ u64 tops[kThreads / 64];
  __shared__ uint32_t lows[kThreads / 64], bads[kThreads / 64];
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.N);
  for (int b = blockIdx.x * kThreads + t; b < kBins; b += gridDim.x * kThreads) {
    a.count[m * kBins + b] = 0;
    a.weight[m * kBins + b] = 0;
  }
  if (blockIdx.x == 0 && t == 0) a.listed[m] = 0;
  u64 top = 0;
  uint32_t low = 0xffffffffu, bad = 0;
  for_logits<TYPE, kThreads>(a, m, begin, end, t, [&](float z, int n) {
    top = max(top, entry_of(z, n));
    if (z > -__builtin_inff()) low = min(low, key_of(z));
    bad |= !(z < __builtin_inff());
  });
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    top = max(top, shuffle_xor(top, d));
    low = min(low, (uint32_t)__shfl_xor((int)low, d, 64));
    bad |= (uint32_t)__shfl_xor((int)bad, d, 64);
  }
  if ((t & 63) == 0) tops[t >> 6] = top, lows[t >> 6] = low, bads[t >> 6] = bad;
  __syncthreads();
  if (t != 0) return;
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) {
    top = max(top, tops[w]);
    low = min(low, lows[w]);
    bad |= bads[w];
  }
  a.part[m * a.chunks + blockIdx.x] = SamplePart{top, low, bad};
}

// ---- launch 2: the histograms of tokens and of weights
template <int TYPE>
__global__ __launch_bounds__(kThreads) void histogram_kernel(SampleArgs a) {
  __shared__ uint32_t count[kBins];
  __shared__ u64 weight[kBins];
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.N);
  for (int b = t; b < kBins; b += kThreads) count[b] = 0, weight[b] = 0;
  const Row r = row_of<kThreads>(a, m, t);  // synchronizes
  if (r.bad || r.greedy) return;            // all of the row's workgroups
  const double least = -(double)(a.bits + 1);
  for_logits<TYPE, kThreads>(a, m, begin, end, t, [&](float z, int) {
    const double d = r.top - (double)z, y = log2_weight(r, d);
    if (!(y >= least)) return;
    const int b = bin_of(r, d);
    atomicAdd(&count[b], 1u);
    atomicAdd(&weight[b], weight_of(y, a.bits));
  });
  __syncthreads();
  for (int b = t; b < kBins; b += kThreads) {
    if (count[b] == 0) continue;
    atomicAdd(a.count + m * kBins + b, count[b]);
    atomicAdd(a.weight + m * kBins + b, weight[b]);
  }
}

// ---- what the histogram says, in launches 3 and 4

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

// Tokens and weights of a row before each bin, with the whole row's behind the last
struct Sums {
  uint32_t count[kBins + 1];
  u64 weight[kBins + 1];
};
// the bins whose tokens are gathered, by bits, and how many tokens they hold
struct Needed {
  uint32_t mask[kBins / 32];
  uint32_t total;
  __device__ bool has(int b) const { return mask[b >> 5] >> (b & 31) & 1; }
};

struct Limits {
  int k;          // 0: none
  double p;       // 1: none
  double y;       // log2 of min_p; below -(bits + 1): none
  double u;
};

__device__ __forceinline__ Limits limits_of(const SampleArgs& a, int64_t m) {
  Limits l;
  const int k = a.top_k ? a.top_k[m] : 0;
  l.k = k > 0 && k < a.N ? k : 0;
  const float p = a.top_p ? a.top_p[m] : 1.0f, q = a.min_p ? a.min_p[m] : 0.0f;
  l.p = p < 1.0f ? fmaxf(p, 0.0f) : 1.0f;
  l.y = q > 0.0f ? log2((double)fminf(q, 1.0f)) : -1e30;
  const float u = a.u[m];
  l.u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
  return l;
}

// where a sum's bounds [lo, hi] put the place that it decides
struct Bounds {
  u64 lo, hi;
};

// Reads the row's histogram into s and marks the bins that decide its token.
template <int T>
__device__ __forceinline__ void plan(const SampleArgs& a, const Row& r, const Limits& l, int64_t m,
                                     int t, Sums& s, Needed& n) {
  constexpr int B = kBins / T;
  __shared__ int at[8];
  uint32_t c[B], cs = 0;
  u64 w[B], ws = 0;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    cs += c[i] = a.count[m * kBins + B * t + i];
    ws += w[i] = a.weight[m * kBins + B * t + i];
  }
  uint32_t ci = cs;
  u64 wi = ws;
  scan<T>(ci, wi, t);
  ci -= cs, wi -= ws;
#pragma unroll
  for (int i = 0; i < B; ++i) {
    s.count[B * t + i] = ci, s.weight[B * t + i] = wi;
    ci += c[i], wi += w[i];
  }
  if (t == T - 1) s.count[kBins] = ci, s.weight[kBins] = wi;
  if (t < kBins / 32) n.mask[t] = 0;
  if (t == 0) n.total = 0;
  if (t < 8) at[t] = 0;
  __syncthreads();

  // at[2 i], at[2 i + 1]: the bins of step i's bounds
  const u64 all = s.weight[kBins];
  Bounds k{all, all};
  const bool by_k = l.k > 0 && (uint32_t)l.k < s.count[kBins];
  if (by_k) {
    for (int b = B * t; b < B * t + B; ++b)
      if (s.count[b] < (uint32_t)l.k && s.count[b + 1] >= (uint32_t)l.k) at[0] = b;
    __syncthreads();
    k = Bounds{s.weight[at[0]], s.weight[at[0] + 1]};
  }
  Bounds p = k;
  const bool by_p = l.p > 0.0 && l.p < 1.0;
  if (by_p) {
    const double lo = l.p * (double)k.lo, hi = l.p * (double)k.hi;
    for (int b = B * t; b < B * t + B; ++b) {
      const double before = (double)s.weight[b], past = (double)s.weight[b + 1];
      if (before < lo && past >= lo) at[2] = b;  // (none where lo is 0: bin 0)
      if (before < hi && past >= hi) at[3] = b;
    }
    __syncthreads();
    p = Bounds{s.weight[at[2]], min(s.weight[at[3] + 1], k.hi)};
  } else if (l.p <= 0.0) {
    p.lo = p.hi = 1ull << a.bits;  // the first token alone
  }
  Bounds q = p;
  const bool by_q = l.y >= -(double)(a.bits + 1);
  int q0 = 0, q1 = 0;
  if (by_q) {
    // the bin of that distance; one to either side for the roundings on the way
    const int b = bin_of(r, -l.y / r.rate);
    q0 = max(b - 1, 0), q1 = min(b + 1, kBins - 1);
    q = Bounds{min(p.lo, s.weight[q0]), min(p.hi, s.weight[q1 + 1])};
  }
  {
    const double lo = l.u * (double)q.lo, hi = l.u * (double)q.hi;
    for (int b = B * t; b < B * t + B; ++b) {
      const double before = (double)s.weight[b], past = (double)s.weight[b + 1];
      if (before <= lo && past > lo) at[4] = b;
      if (before <= hi && past > hi) at[5] = b;
    }
    __syncthreads();
  }
  uint32_t mine = 0;
  for (int b = B * t; b < B * t + B; ++b) {
    const bool need = (by_k && b == at[0]) || (by_p && b >= at[2] && b <= at[3]) ||
                      (by_q && b >= q0 && b <= q1) || (b >= at[4] && b <= at[5]);
    if (!need) continue;
    atomicOr(&n.mask[b >> 5], 1u << (b & 31));
    mine += s.count[b + 1] - s.count[b];
  }
  if (mine) atomicAdd(&n.total, mine);
  __syncthreads();
}

// ---- launch 3: the tokens of those bins
template <int TYPE>
__global__ __launch_bounds__(kThreads) void gather_kernel(SampleArgs a) {
  __shared__ Sums s;
  __shared__ Needed need;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.N);
  const Row r = row_of<kThreads>(a, m, t);
  if (r.bad || r.greedy) return;
  plan<kThreads>(a, r, limits_of(a, m), m, t, s, need);
  if (need.total > kList) return;
  const double least = -(double)(a.bits + 1);
  for_logits<TYPE, kThreads>(a, m, begin, end, t, [&](float z, int n) {
    const double d = r.top - (double)z;
    if (!(log2_weight(r, d) >= least) || !need.has(bin_of(r, d))) return;
    // all of them are need.total <= kList
    a.list[m * kList + atomicAdd(a.listed + m, 1u)] = entry_of(z, n);
  });
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
__device__ __forceinline__ Found search(const SampleArgs& a, const Row& r, int64_t m, int t,
                                        Search how, uint32_t k, double to) {
  __shared__ uint32_t count[256], digit, found_before, found_ties;
  __shared__ u64 weight[256], found_sum, found_weight;
  const double least = -(double)(a.bits + 1);
  uint32_t prefix = 0, before = 0;
  u64 sum = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (t < 256) count[t] = 0, weight[t] = 0;
    __syncthreads();
    for_logits<TYPE, kDraw>(a, m, 0, a.N, t, [&](float z, int) {
      const double y = log2_weight(r, r.top - (double)z);
      const uint32_t key = key_of(z);
      if (!(y >= least) || (shift < 24 && key >> (shift + 8) != prefix)) return;
      const int b = 255 - (key >> shift & 255);  // the largest first
      atomicAdd(&count[b], 1u);
      atomicAdd(&weight[b], weight_of(y, a.bits));
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

template <int TYPE>
__global__ __launch_bounds__(kDraw) void draw_kernel(SampleArgs a) {
  constexpr int E = kList / kDraw;
  __shared__ Sums s;
  __shared__ Needed need;
  __shared__ uint32_t start[kBins];  // a needed bin's first place in the list
  __shared__ u64 list[kList], ahead[kList + 1];
  __shared__ u64 found, below;
  __shared__ int which;
  const int t = threadIdx.x;
  const int64_t m = blockIdx.y;
  const Row r = row_of<kDraw>(a, m, t);
  if (r.bad || r.greedy) {
    if (t == 0) {
      a.token[m] = r.bad ? -1 : r.token;
      if (a.logprob) a.logprob[m] = r.bad ? __builtin_nanf("") : 0.0f;
    }
    return;
  }
  const Limits l = limits_of(a, m);
  plan<kDraw>(a, r, l, m, t, s, need);
  const u64 all = s.weight[kBins];
  const bool by_k = l.k > 0 && (uint32_t)l.k < s.count[kBins];
  const bool by_p = l.p > 0.0 && l.p < 1.0, by_q = l.y >= -(double)(a.bits + 1);
  auto finish = [&](int64_t token, float z, u64 whole) {
    a.token[m] = token;
    if (a.logprob)
      a.logprob[m] = (float)(0.6931471805599453 *
                             (log2_weight(r, r.top - (double)z) -
                              (log2((double)whole) - (double)a.bits)));
  };

  if (need.total > kList) {  // all of the workgroup
    u64 whole = all;
    if (by_k) {
      const Found f = search<TYPE>(a, r, m, t, kByCount, (uint32_t)l.k, 0.0);
      whole = f.sum + (l.k - f.before) * f.weight;
    }
    if (by_p) {
      const double to = l.p * (double)whole;
      const Found f = search<TYPE>(a, r, m, t, kBySum, 0, to);
      whole = min(whole, f.sum + place_among(f.sum, f.weight, f.ties, to, false) * f.weight);
    } else if (l.p <= 0.0) {
      whole = 1ull << a.bits;
    }
    if (by_q) {
      if (t == 0) below = 0;
      __syncthreads();
      u64 mine = 0;
      for_logits<TYPE, kDraw>(a, m, 0, a.N, t, [&](float z, int) {
        const double y = log2_weight(r, r.top - (double)z);
        if (y >= l.y) mine += weight_of(y, a.bits);
      });
      atomicAdd(&below, mine);
      __syncthreads();
      whole = min(whole, below);
    }
    const double to = l.u * (double)whole;
    const Found f = search<TYPE>(a, r, m, t, kPastSum, 0, to);
    const uint32_t place = place_among(f.sum, f.weight, f.ties, to, true);
    const int64_t token = index_of<TYPE>(a, m, t, f.key, place);
    if (t == 0) finish(token, value_of(f.key), whole);
    return;
  }

  // the list sorted, in descending order, zeros (no token's entry) behind it
  const int count = (int)need.total;
  int size = 2;
  while (size < count) size *= 2;
  for (int i = t; i < size; i += kDraw) list[i] = i < count ? a.list[m * kList + i] : 0;
  {
    constexpr int B = kBins / kDraw;
    uint32_t c[B], at = 0;
    u64 none = 0;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int b = B * t + i;
      at += c[i] = need.has(b) ? s.count[b + 1] - s.count[b] : 0;
    }
    const uint32_t mine = at;
    scan<kDraw>(at, none, t);
    at -= mine;
#pragma unroll
    for (int i = 0; i < B; ++i) start[B * t + i] = at, at += c[i];
  }
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int i = t; i < size / 2; i += kDraw) {
        const int lo = 2 * (i - (i & (j - 1))) + (i & (j - 1)), hi = lo + j;
        const u64 x = list[lo], y = list[hi];
        if ((x < y) == ((lo & k) == 0)) list[lo] = y, list[hi] = x;
      }
    }
  if (t == 0) found = all, below = 0, which = 0;
  __syncthreads();

  // weights of places E t .. E t + E - 1 of the list, and the sums ahead of them
  u64 w[E], sum = 0;
  int bin[E];
  double y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = E * t + e;
    w[e] = 0, bin[e] = 0, y[e] = 0.0;
    if (i < count) {
      const double d = r.top - (double)value_of((uint32_t)(list[i] >> 32));
      y[e] = log2_weight(r, d);
      bin[e] = bin_of(r, d);
      w[e] = weight_of(y[e], a.bits);
    }
    sum += w[e];
  }
  uint32_t none = 0;
  u64 total = sum;
  scan<kDraw>(none, total, t);
  u64 before = total - sum;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    ahead[E * t + e] = before;
    before += w[e];
  }
  if (t == kDraw - 1) ahead[kList] = before;
  __syncthreads();
  // the sum of all weights of the row ahead of place i
  auto before_place = [&](int e) {
    const int i = E * t + e;
    return s.weight[bin[e]] + (ahead[i] - ahead[start[bin[e]]]);
  };

  u64 whole = all;
  if (by_k) {
    // the k-th token's bin: every thread finds it
    int b = 0;
    for (int step = kBins / 2; step > 0; step /= 2)
      if (s.count[b + step] < (uint32_t)l.k) b += step;
    const uint32_t first = start[b];
    whole = s.weight[b] + ahead[first + (l.k - s.count[b])] - ahead[first];
  }
  if (by_p) {
    const double to = l.p * (double)whole;
    if (t == 0) found = whole;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (E * t + e >= count) break;
      const u64 b = before_place(e);
      if ((double)b < to && (double)(b + w[e]) >= to) found = min(whole, b + w[e]);
    }
    __syncthreads();
    whole = found;
  } else if (l.p <= 0.0) {
    whole = 1ull << a.bits;
  }
  if (by_q) {
    const int q = bin_of(r, -l.y / r.rate), q0 = max(q - 1, 0), q1 = min(q + 1, kBins - 1);
    u64 mine = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (E * t + e < count && bin[e] >= q0 && bin[e] <= q1 && y[e] >= l.y) mine += w[e];
    if (mine) atomicAdd(&below, mine);
    __syncthreads();
    whole = min(whole, s.weight[q0] + below);
  }
  const double to = l.u * (double)whole;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (E * t + e >= count) break;
    const u64 b = before_place(e);
    if ((double)b <= to && (double)(b + w[e]) > to) which = E * t + e;
  }
  __syncthreads();
  if (t == 0) {
    const u64 it = list[which];
    finish((uint32_t)~(uint32_t)it, value_of((uint32_t)(it >> 32)), whole);
  }
}

constexpr int64_t kRows = 1024;  // of a set of launches: bounds the workspace

struct Layout {
  int64_t rows, chunks, chunk;
  size_t weight, list, part, count, listed, bytes;
};

// A row is split until the launch has 1024 workgroups, into parts of 4096 logits at least
Layout layout(int64_t M, int64_t N) {
  Layout l;
  l.rows = M < kRows ? M : kRows;
  int64_t c = ceil_div(1024, l.rows), most = ceil_div(N, 4096);
  if (c > most) c = most;
  l.chunk = ceil_div(ceil_div(N, c), 2048) * 2048;
  l.chunks = ceil_div(N, l.chunk);
  size_t at = 0;
  auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += (size_t)ceil_div(bytes, 256) * 256;
    return here;
  };
  l.weight = take(8 * l.rows * kBins);
  l.list = take(8 * l.rows * kList);
  l.part = take((int64_t)sizeof(SamplePart) * l.rows * l.chunks);
  l.count = take(4 * l.rows * kBins);
  l.listed = take(4 * l.rows);
  l.bytes = at;
  return l;
}

template <int TYPE>
void launch_type(const SampleArgs& a, int rows, hipStream_t st) {
  const dim3 grid((uint32_t)a.chunks, (uint32_t)rows), one(1, (uint32_t)rows);
  top_kernel<TYPE><<<grid, kThreads, 0, st>>>(a);
  histogram_kernel<TYPE><<<grid, kThreads, 0, st>>>(a);
  gather_kernel<TYPE><<<grid, kThreads, 0, st>>>(a);
  draw_kernel<TYPE><<<one, kDraw, 0, st>>>(a);
}

}  // namespace

size_t sample_workspace(int64_t M, int64_t N) { return layout(M, N).bytes; }

int launch_sample(SampleArgs a, int type, int64_t M, void* ws, hipStream_t st) {
  const Layout l = layout(M, a.N);
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.weight = reinterpret_cast<u64*>(p + l.weight);
  a.list = reinterpret_cast<u64*>(p + l.list);
  a.part = reinterpret_cast<SamplePart*>(p + l.part);
  a.count = reinterpret_cast<uint32_t*>(p + l.count);
  a.listed = reinterpret_cast<uint32_t*>(p + l.listed);
  a.chunk = (int)l.chunk;
  a.chunks = (int)l.chunks;
  int log = 0;
  while (((int64_t)1 << log) < a.N) ++log;
  a.bits = 62 - log < 50 ? 62 - log : 50;
  for (int64_t m = 0; m < M; m += l.rows) {
    const int rows = (int)(M - m < l.rows ? M - m : l.rows);
    type == GEMMQ_F32    ? launch_type<GEMMQ_F32>(a, rows, st)
    : type == GEMMQ_BF16 ? launch_type<GEMMQ_BF16>(a, rows, st)
                         : launch_type<GEMMQ_F16>(a, rows, st);
    a.Z = static_cast<const uint8_t*>(a.Z) + l.rows * a.ldz * type_bytes(type);
    if (a.temperature) a.temperature += l.rows;
    if (a.top_k) a.top_k += l.rows;
    if (a.top_p) a.top_p += l.rows;
    if (a.min_p) a.min_p += l.rows;
    a.u += l.rows;
    a.token += l.rows;
    if (a.logprob) a.logprob += l.rows;
  }
  return 0;
}

}  // namespace i8
}  // namespace gemmq
