// One token a row of logits from a given random number, gfx950 (include/gdn.h, gdn_sample).
//
// Weights are whole numbers: w = round(2^S e^((x - m) / T)), the exponential in 64 bits to 2^-51 of the largest, S = 62 minus
// the bits of the vocabulary's size, at most 51 (44 for 2^18 tokens). Their sums are then exact in any order, atomic or
// not, so a row's token depends on nothing but the row, and a border (top_p's, or the random number's) is met within
// 2^-S of the largest weight a token and a rounding of the sum to 64 bits. Tokens whose weight is 0 do not count at all: they
// come last in the order.
//
// A row is cut into tiles of 512 tokens, a wave each. Without filters two launches over all rows:
//   tiles     the largest value of every tile, and the tile's weight against it: logits are read once
//   choose    (below)
// and with them three or four:
//   extremes  the largest and the least finite value of every tile
//   weigh     rows without top_k and top_p: the weight of every tile. Others: counts and weights of 1024 bins of the distance
//             from the row's largest value, in LDS, then added to the row's
//   gather    (only where top_k or top_p is given) from the bins, the few in which their borders must lie; the weight of every
//             tile's tokens before them, and a list of the tokens inside them
//   choose    a workgroup a row: the list sorted by (value, index), the borders met exactly, the kept ones' weights added to their
//             tiles', the tile in which the weight passes u times the sum, and the token in it
// A kept token is one whose (value, index), as one number that falls with the value and rises with the index, is not
// above the last kept one's. A list that would be longer than 4096 (thousands of equal values at a border) is not made:
// choose then looks the borders up in the row itself, 11 bits of the key at a time.
//
// What bounds it: without filters the vector units (26 instructions a token, 11 of them in 64 bits: 1024 rows of 131072 bf16
// 120 us, where reading them takes 44 to 54; 64-bit exponentials by a longer series and a table of 8: 165). With filters, 64
// rows of 99991 fp32, 6 + 13 + 14 + 8 us: each pass's beginning (the row's ends, the bins' sums) and the weights; one row of 131072 3 + 5
// + 6 + 6 us: dependent launches. Bins are as wide as the row: a mask of large negative numbers in place of minus infinity makes them
// wider and the list longer (131072 tokens, top_p alone: 34 us against 23). Rows without a list are one workgroup's, which reads them
// up to nine times: 131072 equal values 0.80 ms with top_p, 0.37 with top_k, 2^20 of them 6.2 and 2.8 ms, whatever the
// number of rows up to one a CU. Weights of bins only up to the border that a workgroup's own counts give top_k (13.7
// against 12.8 us for weigh) cost more than they saved.

#include <type_traits>

#include "device_common.h"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / kWave;
constexpr int kTile = 8 * kWave;  // tokens of a wave
constexpr int kBins = 1024;
constexpr int kList = 4096;
constexpr uint32_t kLowest = 0x007FFFFFu;  // key_of(-infinity)

// ------------------------------------------------------------------- values and weights

// a key that sorts as the value does
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x == x)) return kLowest;  // a NaN is a token that cannot come
  x += 0.0f;                      // (-0 is 0)
  const uint32_t u = __float_as_uint(x);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
template <typename T>
__device__ __forceinline__ float get(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}

typedef float uf32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t uu32x4 __attribute__((ext_vector_type(4), aligned(2)));

// values [i, i + 8) of a row, minus infinity past its end
template <typename T>
__device__ __forceinline__ void load8(const T* x, int i, int n, float (&v)[8]) {
  if (i + 8 <= n) {
    if constexpr (sizeof(T) == 2) {
      const uu32x4 r = *reinterpret_cast<const uu32x4*>(x + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(r[e] << 16);
        v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
      }
    } else {
      const uf32x4 a = *reinterpret_cast<const uf32x4*>(x + i), b = *reinterpret_cast<const uf32x4*>(x + i + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i + e < n ? get(x + i + e) : -__builtin_inff();
  }
}

// 2^(j / 32) times 2^S, j < 32: the 32 lie in 32 pairs of LDS banks, so that reads of any of them do not meet.
constexpr int kSteps = 32;
__device__ __forceinline__ void fill_steps(double* steps, int shift) {
  if (threadIdx.x < kSteps) {  // the series of e^(j ln 2 / 32); the first term left out is under 2^-56
    const double f = threadIdx.x * (0.693147180559945309417 / kSteps);
    double s = 1.0;
#pragma unroll
    for (int n = 18; n > 0; --n) s = fma(s, f * (1.0 / n), 1.0);
    steps[threadIdx.x] = ldexp(s, shift);
  }
}

enum Mode { kNone, kLikeliest, kPlain, kListed };

// What a row's tokens are judged by.
struct Row {
  float most;          // the largest value; 0 where that is an infinity, whose tokens then have 0 and all others minus infinity
  bool infinite;
  double base;         // most
  double per;          // 32 log2(e) / T
  double low;          // 32 log2 of what is surely rounded to 0
  float far;           // a distance from the largest value beyond which a weight is surely 0 (infinite T: all are nearer)
  float bins;          // bins by distance
  double least;        // 2^S min_p, min_p at most 1
  const double* steps;
  int shift;           // S
  int32_t k;           // 0: no top_k
  float p;             // 1: no top_p
  int mode;            // kNone, kLikeliest, kPlain, or kListed for rows with top_k or top_p

  __device__ __forceinline__ void against(float largest) {
    infinite = largest == __builtin_inff();
    most = infinite ? 0.f : largest;
    base = most;
  }
  __device__ __forceinline__ float seen(float x) const { return !infinite ? x : x == __builtin_inff() ? 0.f : -__builtin_inff(); }
  template <int N>
  __device__ __forceinline__ void see(float (&v)[N]) const {
    if (infinite) {  // (the row agrees)
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = seen(v[e]);
    }
  }
  // 2^S e^((x - most) / T): t = 32 log2 of the exponential, its nearest whole number n and the rest f, |f| <= 1/2;
  // 2^(t / 32) = 2^(n / 32) e^z, z = f ln 2 / 32, by the series to z^5 with z^6 / 720 taken into z^2 and z^4 (economised: on |z| <= a it
  // is a^4 (3/2 (z/a)^2 - 9/16) z^2 / 720 to a^6 / 11520). Good to 2^-51.8, and a weight, with what t loses, to 2^-51 of the largest.
  // (A NaN, also from minus infinity at an infinite T, is dropped by the largest of it and `low`.)
  __device__ __forceinline__ double weight(float x) const {
    constexpr double c = 0.693147180559945309417 / kSteps, a = c / 2;
    constexpr double c2 = 1.0 / 2.0 - 9.0 / 16.0 * a * a * a * a / 720.0, c4 = 1.0 / 24.0 + 3.0 / 2.0 * a * a / 720.0;
    const double t = __builtin_fmax((static_cast<double>(x) - base) * per, low);
    const double whole = t + 0x1.8p52;
    const int n = static_cast<int>(__double_as_longlong(whole));
    const double f = t - (whole - 0x1.8p52);
    double s = fma(f, c * c * c * c * c / 120.0, c4 * c * c * c * c);
    s = fma(s, f, c * c * c / 6.0);
    s = fma(s, f, c2 * c * c);
    s = fma(s, f, c);
    s = fma(s, f, 1.0);
    const double step = steps[n & (kSteps - 1)];
    return s * __hiloint2double(__double2hiint(step) + ((n & ~(kSteps - 1)) << 15), __double2loint(step));
  }
  // rounded: the low bits of 2^52 + w
  __device__ __forceinline__ static unsigned long long whole(double w) {
    return __double_as_longlong(w + 0x1p52) & 0xFFFFFFFFFFFFFull;
  }
  // -1: no token that could come
  __device__ __forceinline__ int bin(float x) const {
    const float d = most - x;
    const int b = static_cast<int>(fminf(d * bins, kBins - 1.0f));
    return d <= far && x > -__builtin_inff() ? b : -1;
  }
};
// the sum of eight tokens' weights, rounded (the bits of 2^52 + w, less those of the eight 2^52)
__device__ __forceinline__ unsigned long long sum_of(const Row& row, const float (&v)[8]) {
  unsigned long long sum = 0 - 8 * 0x4330000000000000ull;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum += __double_as_longlong(row.weight(v[e]) + 0x1p52);
  return sum;
}

// the order of tokens: lower numbers first
__device__ __forceinline__ unsigned long long place_of(float x, int i) {
  return static_cast<unsigned long long>(~key_of(x)) << 32 | static_cast<uint32_t>(i);
}

// ------------------------------------------------------------------------ the workspace

struct Plan {  // of a row with a filter, from gather to choose
  int32_t looked;   // the list is not made
  int32_t count;    // tokens in the list
  int32_t top;      // the bin of top_k's border (kBins: none), and how many tokens of it stay
  uint32_t stay;
  int32_t from, to;  // the bins between which top_p's border lies (none: from > to)
  unsigned long long whole;   // the weight of the bins before `top`
  unsigned long long before;  // the weight of the bins before `from`
};

struct Space {
  uint2* ends;                 // [rows][tiles] largest and least key
  unsigned long long* sums;    // [rows][tiles]
  unsigned long long* weights; // [rows][kBins]
  uint32_t* counts;            // [rows][kBins]
  uint32_t* listed;            // [rows]
  Plan* plans;                 // [rows]
  uint32_t* list;              // [rows][kList]
};

struct Call {
  SampleArgs a;
  Space w;
  int tiles;   // of a row
  int groups;  // workgroups a row in weigh and gather
  int shift;
  int first;   // the launch's first row
};

// Lane operations along rows of 16 lanes, then over the rows (DPP): lane 63 has seen all.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(none), static_cast<int>(v), CTRL, ROWS, 0xF, false));
}
template <typename F>
__device__ __forceinline__ uint32_t wave_all(uint32_t v, uint32_t none, F join) {
  v = join(v, moved<0x111, 0xF>(v, none));
  v = join(v, moved<0x112, 0xF>(v, none));
  v = join(v, moved<0x114, 0xF>(v, none));
  v = join(v, moved<0x118, 0xF>(v, none));
  v = join(v, moved<0x142, 0xA>(v, none));
  v = join(v, moved<0x143, 0xC>(v, none));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), kWave - 1));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_all(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  return wave_all(v, 0xFFFFFFFFu, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int CTRL, int ROWS>
__device__ __forceinline__ unsigned long long add_moved(unsigned long long v) {
  const uint32_t lo = moved<CTRL, ROWS>(static_cast<uint32_t>(v), 0), hi = moved<CTRL, ROWS>(static_cast<uint32_t>(v >> 32), 0);
  return v + (static_cast<unsigned long long>(hi) << 32 | lo);
}
// the sum over the lanes up to each one
__device__ __forceinline__ unsigned long long wave_scan(unsigned long long v) {
  v = add_moved<0x111, 0xF>(v);
  v = add_moved<0x112, 0xF>(v);
  v = add_moved<0x114, 0xF>(v);
  v = add_moved<0x118, 0xF>(v);
  v = add_moved<0x142, 0xA>(v);
  return add_moved<0x143, 0xC>(v);
}

// Sum over the threads up to each one; `all` gets the sum of all.
struct Scan {
  unsigned long long part[2][kWaves];
};
__device__ __forceinline__ unsigned long long scan(unsigned long long v, Scan& s, int& turn, unsigned long long& all) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  v = wave_scan(v);
  turn ^= 1;  // (the readers of the last turn's parts need not be done)
  if (lane == kWave - 1) s.part[turn][w] = v;
  __syncthreads();
  all = 0;
  unsigned long long before = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) before = all;
    all += s.part[turn][i];
  }
  return v + before;
}

// Two such sums at once, of counts and of weights. (No sum of either kind may follow before the next barrier.)
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += moved<0x111, 0xF>(v, 0);
  v += moved<0x112, 0xF>(v, 0);
  v += moved<0x114, 0xF>(v, 0);
  v += moved<0x118, 0xF>(v, 0);
  v += moved<0x142, 0xA>(v, 0);
  return v + moved<0x143, 0xC>(v, 0);
}
__device__ __forceinline__ void scan(uint32_t n, unsigned long long v, Scan& s, uint32_t& upto_n, unsigned long long& upto_v,
                                     uint32_t& all_n, unsigned long long& all_v) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  upto_n = wave_scan(n);
  upto_v = wave_scan(v);
  if (lane == kWave - 1) {
    s.part[0][w] = upto_n;
    s.part[1][w] = upto_v;
  }
  __syncthreads();
  all_n = 0;
  all_v = 0;
  uint32_t before_n = 0;
  unsigned long long before_v = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) {
      before_n = all_n;
      before_v = all_v;
    }
    all_n += static_cast<uint32_t>(s.part[0][i]);
    all_v += s.part[1][i];
  }
  upto_n += before_n;
  upto_v += before_v;
}

// What a row's parameters ask for: formed by one lane, for all after the next barrier.
struct Asked {
  double per, least;
  float far, p;
  int32_t k;
  int mode;
};
__device__ __forceinline__ void ask(const Call& c, int r, Asked& to) {
  if (threadIdx.x != kThreads - 1) return;  // (its wave has no part in fill_steps)
  const float t = c.a.temperature ? c.a.temperature[r] : 1.0f;
  const float min_p = c.a.min_p ? c.a.min_p[r] : 0.f;
  const int32_t k = c.a.top_k ? c.a.top_k[r] : 0;
  const float p = c.a.top_p ? c.a.top_p[r] : 1.f;
  to.per = 1.44269504088896340736 * kSteps / static_cast<double>(t);
  to.far = t * (0.693147180559945309417f * (c.shift + 1.5f));
  to.least = ldexp(min_p > 0.f ? (min_p < 1.f ? min_p : 1.0) : 0.0, c.shift);
  to.k = k < 0 || k >= c.a.vocab ? 0 : k;
  to.p = p < 1.f ? p : 1.f;
  to.mode = !(t > 0.f) ? kLikeliest : to.k == 0 && to.p == 1.f ? kPlain : kListed;
}
__device__ __forceinline__ Row asked(const Call& c, const Asked& from, const double* steps) {
  Row row{};
  row.per = from.per;
  row.far = from.far;
  row.least = from.least;
  row.k = from.k;
  row.p = from.p;
  row.mode = from.mode;
  row.shift = c.shift;
  row.low = -kSteps * (c.shift + 12.0);  // (a tile of 512 such tokens is rounded to 0 too)
  row.steps = steps;
  return row;
}

// The row's largest and least values, and what its parameters ask for. Every thread gets it.
struct Ends {
  uint32_t part[2][kWaves];
  Asked asked;
};
__device__ __forceinline__ Row row_of(const Call& c, int r, const double* steps, Ends& sh) {
  uint32_t most = 0, least = 0xFFFFFFFFu;
  const uint2* e = c.w.ends + static_cast<int64_t>(r) * c.tiles;
  ask(c, r, sh.asked);
  for (int t = threadIdx.x; t < c.tiles; t += kThreads) {
    const uint2 x = e[t];
    most = max(most, x.x);
    least = min(least, x.y);
  }
  most = wave_max(most);
  least = wave_min(least);
  if (threadIdx.x % kWave == 0) {
    sh.part[0][threadIdx.x / kWave] = most;
    sh.part[1][threadIdx.x / kWave] = least;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    most = max(most, sh.part[0][w]);
    least = min(least, sh.part[1][w]);
  }
  Row row = asked(c, sh.asked, steps);
  row.against(value_of(most));
  const float range = row.infinite ? 0.f : fminf(row.most - value_of(least), row.far);
  row.bins = range > 0.f ? fminf(kBins * __builtin_amdgcn_rcpf(range), 1e30f) : 0.f;
  if (most <= kLowest) row.mode = kNone;
  return row;
}

// -------------------------------------------------------------------------- extremes

__device__ __forceinline__ uint2 ends_of(const float (&v)[8]) {
  uint32_t most = kLowest, least = 0xFFFFFFFFu;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t k = key_of(v[e]);
    most = max(most, k);
    least = min(least, k > kLowest ? k : 0xFFFFFFFFu);
  }
  return uint2{wave_max(most), wave_min(least)};
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_extremes_kernel(Call c) {
  const int r = c.first + blockIdx.x / c.groups, g = blockIdx.x % c.groups;
  const int lane = threadIdx.x & (kWave - 1);
  if (c.w.counts && g == 0) {  // the row's bins and list begin empty
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      c.w.counts[static_cast<int64_t>(r) * kBins + i] = 0;
      c.w.weights[static_cast<int64_t>(r) * kBins + i] = 0;
    }
    if (threadIdx.x == 0) c.w.listed[r] = 0;
  }
  const T* x = static_cast<const T*>(c.a.logits) + r * c.a.stride;
  uint2* to = c.w.ends + static_cast<int64_t>(r) * c.tiles;
  const int step = c.groups * kWaves;
  for (int t = g * kWaves + threadIdx.x / kWave; t < c.tiles; t += 2 * step) {
    float v[2][8];
    load8(x, t * kTile + 8 * lane, c.a.vocab, v[0]);
    load8(x, min(t + step, c.tiles - 1) * kTile + 8 * lane, c.a.vocab, v[1]);
    const uint2 a = ends_of(v[0]), b = ends_of(v[1]);
    if (lane == 0) to[t] = a;
    if (lane == 0 && t + step < c.tiles) to[t + step] = b;
  }
}

// ------------------------------------------------------------------------------ tiles

// The tile's largest value and its weight against that.
template <typename T>
__global__ __launch_bounds__(kThreads) void sample_tiles_kernel(Call c) {
  __shared__ double steps[kSteps];
  const int r = c.first + blockIdx.x / c.groups, g = blockIdx.x % c.groups;
  const int lane = threadIdx.x & (kWave - 1);
  __shared__ Asked sh;
  fill_steps(steps, c.shift);
  ask(c, r, sh);
  __syncthreads();
  Row row = asked(c, sh, steps);
  const T* x = static_cast<const T*>(c.a.logits) + r * c.a.stride;
  const int step = c.groups * kWaves;
  float v[8], next[8];
  int t = g * kWaves + threadIdx.x / kWave;
  if (t < c.tiles) load8(x, t * kTile + 8 * lane, c.a.vocab, next);
  for (; t < c.tiles; t += step) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    load8(x, min(t + step, c.tiles - 1) * kTile + 8 * lane, c.a.vocab, next);
    float top = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, v[e]);  // (of a NaN and a number: the number)
    const uint32_t most = wave_max(key_of(top));
    unsigned long long sum = 0;
    if (row.mode == kPlain && most > kLowest) {
      row.against(value_of(most));
      row.see(v);
      sum = wave_scan(sum_of(row, v));
    }
    if (lane == kWave - 1) {
      c.w.ends[static_cast<int64_t>(r) * c.tiles + t] = uint2{most, 0xFFFFFFFFu};
      c.w.sums[static_cast<int64_t>(r) * c.tiles + t] = sum;
    }
  }
}

// ------------------------------------------------------------------------------ weigh

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_weigh_kernel(Call c) {
  __shared__ unsigned long long weights[kBins];
  __shared__ uint32_t counts[kBins];
  __shared__ Ends ends;
  __shared__ double steps[kSteps];
  const int r = c.first + blockIdx.x / c.groups, g = blockIdx.x % c.groups;
  const int lane = threadIdx.x & (kWave - 1), step = c.groups * kWaves;
  const T* x = static_cast<const T*>(c.a.logits) + r * c.a.stride;
  int t = g * kWaves + threadIdx.x / kWave;
  float v[8], next[8];
  if (t < c.tiles) load8(x, t * kTile + 8 * lane, c.a.vocab, next);
  fill_steps(steps, c.shift);
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    weights[i] = 0;
    counts[i] = 0;
  }
  const Row row = row_of(c, r, steps, ends);  // (with a barrier)
  if (row.mode < kPlain) return;
  const bool plain = row.mode == kPlain, heavy = row.p < 1.f;
  for (; t < c.tiles; t += step) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    load8(x, min(t + step, c.tiles - 1) * kTile + 8 * lane, c.a.vocab, next);
    row.see(v);
    if (plain) {
      unsigned long long sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const double w = row.weight(v[e]);
        sum += w < row.least ? 0 : row.whole(w);
      }
      sum = wave_scan(sum);
      if (lane == kWave - 1) c.w.sums[static_cast<int64_t>(r) * c.tiles + t] = sum;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int b = row.bin(v[e]);
        if (b >= 0) atomicAdd(&counts[b], 1u);
        if (heavy) {  // (top_k alone needs no weights of bins)
          const unsigned long long w = row.whole(row.weight(v[e]));
          if (b >= 0) atomicAdd(&weights[b], w);
        }
      }
    }
  }
  if (plain) return;
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    if (counts[i]) atomicAdd(&c.w.counts[static_cast<int64_t>(r) * kBins + i], counts[i]);
    if (weights[i]) atomicAdd(&c.w.weights[static_cast<int64_t>(r) * kBins + i], weights[i]);
  }
}

// ----------------------------------------------------------------------------- gather

// f(value, whether the lane has one) for the tokens of a lane's bits, one at a time, as many times as the lane with most of them
// has.
template <typename F>
__device__ __forceinline__ void each_of(uint32_t some, const float (&v)[8], F f) {
  float own[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    own[q] = v[q];
    asm("" : "+v"(own[q]));  // (in registers: else the choice below becomes an address)
  }
  while (__ballot(some != 0)) {
    const int e = __builtin_ctz(some | 0x100u);
    float y = own[0];
#pragma unroll
    for (int q = 1; q < 8; ++q) y = e == q ? own[q] : y;
    f(y, some != 0);
    some &= some - 1;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_gather_kernel(Call c) {
  static_assert(kBins == 2 * kThreads, "two bins a thread");
  __shared__ Scan parts;
  __shared__ Ends ends;
  __shared__ double steps[kSteps];
  __shared__ uint32_t found[kList], n_found, found_at;  // the workgroup's part of the list
  __shared__ int top_at, from_at, to_at;
  __shared__ unsigned long long whole_at, most_at, before_at;
  __shared__ uint32_t stay_at;
  const int r = c.first + blockIdx.x / c.groups, g = blockIdx.x % c.groups;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), step = c.groups * kWaves;
  const T* x = static_cast<const T*>(c.a.logits) + r * c.a.stride;
  int t = g * kWaves + tid / kWave;
  float v[8], next[8];
  if (t < c.tiles) load8(x, t * kTile + 8 * lane, c.a.vocab, next);
  // the bins' counts and weights, and those of all bins before them
  uint32_t n2[2], nb[2], all_n;
  unsigned long long w2[2], wb[2], all_w;
  {
    const uint2 n = *reinterpret_cast<const uint2*>(c.w.counts + static_cast<int64_t>(r) * kBins + 2 * tid);
    const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(c.w.weights + static_cast<int64_t>(r) * kBins + 2 * tid);
    n2[0] = n.x;
    n2[1] = n.y;
    w2[0] = w.x;
    w2[1] = w.y;
  }
  fill_steps(steps, c.shift);
  const Row row = row_of(c, r, steps, ends);
  if (row.mode != kListed) return;
  int turn = 0;
  scan(n2[0] + n2[1], w2[0] + w2[1], parts, nb[0], wb[0], all_n, all_w);
  nb[0] -= n2[0] + n2[1];
  wb[0] -= w2[0] + w2[1];
  nb[1] = nb[0] + n2[0];
  wb[1] = wb[0] + w2[0];
  const bool by_count = row.k > 0 && static_cast<uint32_t>(row.k) < all_n, by_weight = row.p < 1.f;
  if (tid == 0) {
    from_at = to_at = 0;
    before_at = 0;
    n_found = 0;
    if (!by_count) {
      top_at = kBins;
      stay_at = 0;
      whole_at = most_at = all_w;
    }
  }
  if (by_count) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (nb[e] < static_cast<unsigned>(row.k) && static_cast<unsigned>(row.k) <= nb[e] + n2[e]) {
        top_at = 2 * tid + e;
        stay_at = static_cast<uint32_t>(row.k - nb[e]);
        whole_at = wb[e];
        most_at = wb[e] + w2[e];  // (of the bin of top_k's border a part stays)
      }
  }
  __syncthreads();
  const int top = top_at;
  if (by_weight) {
    const double low = static_cast<double>(row.p) * static_cast<double>(whole_at);
    const double high = static_cast<double>(row.p) * static_cast<double>(most_at);
    // the last bin before which too little lies, for either
    int a = -1, b = -1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (n2[e] == 0 || 2 * tid + e > top) continue;
      if (static_cast<double>(wb[e]) < low) a = 2 * tid + e;
      if (static_cast<double>(wb[e]) < high) b = 2 * tid + e;
    }
    const int wa = static_cast<int>(wave_max(static_cast<uint32_t>(a + 1))), wb1 = static_cast<int>(wave_max(static_cast<uint32_t>(b + 1)));
    if (lane == 0 && wa) atomicMax(&from_at, wa - 1);
    if (lane == 0 && wb1) atomicMax(&to_at, wb1 - 1);
    __syncthreads();
  }
  const int from = by_weight ? from_at : kBins, to = by_weight ? to_at : -1;
  const int sure = by_weight ? from : top;  // bins before this one stay
  unsigned long long mine = 0, inside;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int b = 2 * tid + e;
    if (by_weight && b == from) before_at = wb[e];
    if ((b >= from && b <= to) || b == top) mine += n2[e];
  }
  scan(mine, parts, turn, inside);
  const bool looked = inside > kList;
  if (g == 0 && tid == 0)
    c.w.plans[r] = Plan{looked, static_cast<int32_t>(looked ? 0 : inside), top, stay_at, from, to, whole_at, before_at};
  if (looked) return;
  for (; t < c.tiles; t += step) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    load8(x, min(t + step, c.tiles - 1) * kTile + 8 * lane, c.a.vocab, next);
    row.see(v);
    const int i0 = t * kTile + 8 * lane;
    uint32_t stays = 0, listed = 0;  // bits of the lane's tokens
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int b = row.bin(v[e]);
      stays |= (b >= 0 && b < sure) << e;
      listed |= ((b >= from && b <= to) || b == top) << e;
    }
    unsigned long long sum = 0;  // (few stay, mostly)
    each_of(stays, v, [&](float y, bool there) {
      const double w = row.weight(y);
      sum += !there || w < row.least ? 0 : row.whole(w);
    });
    if (listed) {
      uint32_t at = atomicAdd(&n_found, static_cast<uint32_t>(__builtin_popcount(listed)));
      while (listed) {
        if (at < kList) found[at] = i0 + __builtin_ctz(listed);
        ++at;
        listed &= listed - 1;
      }
    }
    sum = wave_scan(sum);
    if (lane == kWave - 1) c.w.sums[static_cast<int64_t>(r) * c.tiles + t] = sum;
  }
  __syncthreads();
  if (tid == 0 && n_found) found_at = atomicAdd(&c.w.listed[r], n_found);
  __syncthreads();
  for (uint32_t i = tid; i < n_found; i += kThreads)
    if (found_at + i < kList) c.w.list[static_cast<int64_t>(r) * kList + found_at + i] = found[i];
}

// ----------------------------------------------------------------------------- choose

struct Choose {
  union {
    unsigned long long list[kList];
    struct {  // the lookup
      uint32_t count[2048];
      unsigned long long weight[2048];
    } look;
  };
  Scan parts;
  Ends ends;
  double steps[kSteps];
  unsigned long long wide;
  uint32_t at;
};

// Where a filter's order ends: every key above `key`, and of the equal ones the first `equal` by index.
struct Border {
  uint32_t key;
  uint32_t equal;
};

// The border of the first `want` tokens (BY_COUNT), or of those before which less than `target` of weight lies, among the tokens
// up to `limit`, from the row itself: counts or weights by the key's leading 11 bits, the next 11 inside the one found, the last 10.
template <typename T, bool BY_COUNT>
__device__ Border look_up(const T* x, int vocab, const Row& row, const Border& limit, uint32_t want, double target, Choose& sh, int& turn) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0;
  unsigned long long before = 0;  // count or weight of the keys above those bits
  uint32_t found = 0;
  int left = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11, bins = 1 << bits, low = left - bits;
    __syncthreads();
    for (int b = tid; b < 2048; b += kThreads) {
      sh.look.count[b] = 0;
      sh.look.weight[b] = 0;
    }
    if (tid == 0) sh.wide = 0;
    __syncthreads();
    for (int i0 = 8 * tid; i0 < vocab; i0 += 8 * kThreads) {
      float v[8];
      load8(x, i0, vocab, v);
      row.see(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (row.bin(v[e]) < 0) continue;
        const uint32_t key = key_of(v[e]);
        if (key < limit.key || (level > 0 && (key >> left) != prefix)) continue;
        const uint32_t b = (key >> low) & (bins - 1);
        atomicAdd(&sh.look.count[b], 1u);
        if (!BY_COUNT && key > limit.key) atomicAdd(&sh.look.weight[b], row.whole(row.weight(v[e])));
      }
    }
    __syncthreads();
    if (!BY_COUNT && tid == 0 && limit.key != 0 && (level == 0 || (limit.key >> left) == prefix))
      sh.look.weight[(limit.key >> low) & (bins - 1)] += limit.equal * row.whole(row.weight(value_of(limit.key)));
    __syncthreads();
    // four bins a thread, from the highest; the last with anything in it before which too little lies
    unsigned long long n[4], sum = 0, all;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = bins - 1 - (4 * tid + e);
      n[e] = b < 0 ? 0 : BY_COUNT ? sh.look.count[b] : sh.look.weight[b];
      sum += n[e];
    }
    unsigned long long at = before + scan(sum, sh.parts, turn, all) - sum;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int b = bins - 1 - (4 * tid + e);
      // (bins lie below 2^11, so a later one is a larger number: its place from the top, plus one)
      if (b >= 0 && sh.look.count[b] && (BY_COUNT ? at < want : static_cast<double>(at) < target)) atomicMax(&sh.wide, bins - static_cast<unsigned long long>(b));
      at += n[e];
    }
    __syncthreads();
    if (sh.wide == 0) {  // (a target of 0: the first of all)
      __syncthreads();
#pragma unroll
      for (int e = 3; e >= 0; --e) {
        const int b = bins - 1 - (4 * tid + e);
        if (b >= 0 && sh.look.count[b]) atomicMax(&sh.wide, 4096ull + b);
      }
      __syncthreads();
    }
    const unsigned long long hit = sh.wide;
    const int b = static_cast<int>(hit >= 4096 ? hit - 4096 : bins - hit);
    // what lies before it
    unsigned long long above = 0;
    for (int q = b + 1 + tid; q < bins; q += kThreads) above += BY_COUNT ? sh.look.count[q] : sh.look.weight[q];
    scan(above, sh.parts, turn, all);
    before += all;
    found = sh.look.count[b];
    prefix = level == 0 ? b : (prefix << bits) | b;
    left = low;
  }
  __syncthreads();
  Border out{prefix, found};
  if (out.key == limit.key) out.equal = min(out.equal, limit.equal);
  if (BY_COUNT) {
    out.equal = min(out.equal, static_cast<uint32_t>(want - before));
  } else {
    const unsigned long long w = row.whole(row.weight(value_of(out.key)));
    uint32_t lo = 1, hi = out.equal;  // the largest j with before + (j - 1) w < target, at least 1
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      if (static_cast<double>(before + (mid - 1) * w) < target) lo = mid;
      else hi = mid - 1;
    }
    out.equal = lo;
  }
  return out;
}

// The place of the last token up to a border: the equal-th in index order of those with its key.
template <typename T>
__device__ unsigned long long last_place(const T* x, int vocab, const Row& row, const Border& b, Choose& sh, int& turn) {
  unsigned long long seen = 0, all;
  __syncthreads();
  if (threadIdx.x == 0) sh.at = 0xFFFFFFFFu;
  for (int i0 = 0; i0 < vocab; i0 += 8 * kThreads) {
    const int i = i0 + 8 * threadIdx.x;
    float v[8];
    load8(x, i, vocab, v);
    row.see(v);
    unsigned long long mine = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mine += i + e < vocab && key_of(v[e]) == b.key;
    unsigned long long at = seen + scan(mine, sh.parts, turn, all) - mine;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < vocab && key_of(v[e]) == b.key && ++at == b.equal) sh.at = i + e;
    seen += all;
    if (seen >= b.equal) break;
  }
  __syncthreads();
  return static_cast<unsigned long long>(~b.key) << 32 | sh.at;
}

// TILES: the weights are the tiles' own, each against its largest value.
template <typename T, bool TILES>
__global__ __launch_bounds__(kThreads) void sample_choose_kernel(Call c) {
  __shared__ Choose sh;
  extern __shared__ unsigned long long tiles[];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave, r = c.first + blockIdx.x, vocab = c.a.vocab;
  const T* x = static_cast<const T*>(c.a.logits) + r * c.a.stride;
  Plan plan{};  // (what is read of a row without one goes nowhere)
  int32_t listed = 0;
  if (!TILES && c.w.counts) {
    plan = c.w.plans[r];
    listed = c.w.list[static_cast<int64_t>(r) * kList + tid];
  }
  fill_steps(sh.steps, c.shift);
  Row row = row_of(c, r, sh.steps, sh.ends);
  const auto answer = [&](int token, float prob) {
    c.a.tokens[r] = token;
    if (c.a.prob) c.a.prob[r] = prob;
  };
  if (row.mode == kNone) {
    if (tid == 0) answer(-1, 0.f);
    return;
  }
  if (row.mode == kLikeliest) {
    if (tid == 0) sh.at = 0xFFFFFFFFu;
    __syncthreads();
    const uint32_t most = key_of(row.infinite ? __builtin_inff() : row.most);
    for (int t = tid; t < c.tiles; t += kThreads)
      if (c.w.ends[static_cast<int64_t>(r) * c.tiles + t].x == most) {
        atomicMin(&sh.at, static_cast<uint32_t>(t));
        break;
      }
    __syncthreads();
    const int i0 = sh.at * kTile;
    __syncthreads();
    if (tid == 0) sh.at = 0xFFFFFFFFu;
    __syncthreads();
    for (int i = i0 + tid; i < min(i0 + kTile, vocab); i += kThreads)
      if (key_of(get(x + i)) == most) atomicMin(&sh.at, static_cast<uint32_t>(i));
    __syncthreads();
    if (tid == 0) answer(sh.at, 1.f);
    return;
  }
  int turn = 0;
  unsigned long long end = ~0ull;  // the last kept token's place
  const auto kept = [&](float v, int i) -> unsigned long long {
    const double f = row.weight(v);
    return place_of(v, i) > end || f < row.least ? 0 : row.whole(f);
  };
  if (!TILES && row.mode == kListed && plan.looked) {
    Border border{0, 0xFFFFFFFFu};
    if (row.k > 0) {
      unsigned long long n = 0, all;
      for (int i = tid; i < kBins; i += kThreads) n += c.w.counts[static_cast<int64_t>(r) * kBins + i];
      scan(n, sh.parts, turn, all);
      if (static_cast<unsigned long long>(row.k) < all) border = look_up<T, true>(x, vocab, row, border, row.k, 0.0, sh, turn);
    }
    if (row.p < 1.f) {
      unsigned long long n = 0, all;
      const bool cut = border.key != 0;
      for (int i0 = 8 * tid; i0 < vocab; i0 += 8 * kThreads) {
        float v[8];
        load8(x, i0, vocab, v);
        row.see(v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!cut || key_of(v[e]) > border.key) n += row.whole(row.weight(v[e]));
      }
      scan(n, sh.parts, turn, all);
      if (cut) all += border.equal * row.whole(row.weight(value_of(border.key)));
      border = look_up<T, false>(x, vocab, row, border, 0, static_cast<double>(row.p) * static_cast<double>(all), sh, turn);
    }
    if (border.key != 0) end = last_place(x, vocab, row, border, sh, turn);
    for (int t = w; t < c.tiles; t += kWaves) {
      unsigned long long sum = 0;
      float v[8];
      const int i0 = t * kTile + 8 * lane;
      load8(x, i0, vocab, v);
      row.see(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += kept(v[e], i0 + e);
      sum = wave_scan(sum);
      if (lane == kWave - 1) tiles[t] = sum;
    }
    __syncthreads();
  } else {
    for (int t = tid; t < c.tiles; t += kThreads) {
      unsigned long long sum = c.w.sums[static_cast<int64_t>(r) * c.tiles + t];
      if (TILES && sum) {  // against the row's largest value
        const double f = row.weight(row.seen(value_of(c.w.ends[static_cast<int64_t>(r) * c.tiles + t].x)));
        sum = static_cast<unsigned long long>(rint(static_cast<double>(sum) * ldexp(f, -c.shift)));
      }
      tiles[t] = sum;
    }
    if (!TILES && row.mode == kListed && plan.count > 0) {
      const auto place = [&](int at) { return place_of(row.seen(get(x + at)), at); };
      if (plan.count <= kThreads) {  // a wave orders its 64; then each one's number is how many of every 64 lie
        // before it (286 entries 1.7 us; each against all others 6 to 8)
        unsigned long long* runs = sh.list + kThreads;
        const unsigned long long mine = tid < plan.count ? place(listed) : 0xFFFFFFFF00000000ull | tid;  // (behind all)
        int before = 0;
#pragma unroll
        for (int l = 0; l < kWave; ++l) {
          const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(mine >> 32), l);
          const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(mine), l);
          before += (static_cast<unsigned long long>(hi) << 32 | lo) < mine;
        }
        runs[w * kWave + before] = mine;
        const auto search = [&](auto n) {
          constexpr int N = decltype(n)::value;
          int at[N] = {};
#pragma unroll
          for (int d = kWave / 2; d > 0; d /= 2)
#pragma unroll
            for (int q = 0; q < N; ++q) at[q] += runs[q * kWave + at[q] + d - 1] < mine ? d : 0;
          before = 0;
#pragma unroll
          for (int q = 0; q < N; ++q) before += at[q] + (runs[q * kWave + at[q]] < mine);
        };
        __syncthreads();
        if (w * kWave < plan.count) {
          if (plan.count > 4 * kWave) search(std::integral_constant<int, 8>{});
          else if (plan.count > 2 * kWave) search(std::integral_constant<int, 4>{});
          else if (plan.count > kWave) search(std::integral_constant<int, 2>{});
          if (tid < plan.count) sh.list[before] = mine;
        }
      } else {
        int size = 2 * kThreads;
        while (size < plan.count) size *= 2;
        for (int i = tid; i < size; i += kThreads) sh.list[i] = i < plan.count ? place(c.w.list[static_cast<int64_t>(r) * kList + i]) : ~0ull;
        // exchanges between partners at falling distances, in runs of rising length
        for (int run = 2; run <= size; run *= 2)
          for (int d = run / 2; d > 0; d /= 2) {
            __syncthreads();
            for (int q = tid; q < size / 2; q += kThreads) {
              const int i = 2 * q - (q & (d - 1)), j = i + d;
              const unsigned long long a = sh.list[i], b = sh.list[j];
              if ((a > b) == ((i & run) == 0)) {
                sh.list[i] = b;
                sh.list[j] = a;
              }
            }
          }
      }
      __syncthreads();
      // up to eight tokens a thread, in order
      const int each = (plan.count + kThreads - 1) / kThreads;
      double wt[8];
      unsigned long long at_top = 0, stays = 0, all;
      int b[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= each) break;
        const int i = each * tid + e;
        b[e] = kBins + 1;
        wt[e] = 0.0;
        if (i < plan.count) {
          const float v = value_of(~static_cast<uint32_t>(sh.list[i] >> 32));
          b[e] = row.bin(v);
          wt[e] = row.weight(v);
          at_top += b[e] < plan.top;
        }
      }
      scan(at_top, sh.parts, turn, all);
      const int stay_end = plan.top < kBins ? static_cast<int>(all) + static_cast<int>(plan.stay) : kBins + kList;
      // (the tokens of top_k's bin come last in the list: those up to stay_end are its)
      unsigned long long mine = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= each) break;
        if (b[e] == plan.top && each * tid + e < stay_end) stays += row.whole(wt[e]);
        if (b[e] <= plan.to) mine += row.whole(wt[e]);
      }
      scan(stays, sh.parts, turn, all);
      const double target = static_cast<double>(row.p) * static_cast<double>(plan.whole + all);
      const bool by_weight = plan.from <= plan.to;
      unsigned long long before = plan.before + scan(mine, sh.parts, turn, all) - mine;
      int last = -1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= each) break;
        const int i = each * tid + e;
        const bool stay = i < plan.count && i < stay_end &&
                          (!by_weight || (b[e] <= plan.to && (static_cast<double>(before) < target || (i == 0 && plan.from == 0))));
        if (b[e] <= plan.to) before += row.whole(wt[e]);
        if (!stay) continue;
        last = i;
        if (!(wt[e] < row.least)) atomicAdd(&tiles[static_cast<uint32_t>(sh.list[i]) / kTile], row.whole(wt[e]));
      }
      if (tid == 0) sh.at = 0;
      __syncthreads();
      const uint32_t most = wave_max(static_cast<uint32_t>(last + 1));
      if (lane == 0 && most) atomicMax(&sh.at, most - 1);
      __syncthreads();
      end = sh.list[sh.at];
    }
    __syncthreads();
  }
  // the tile in which the weight passes the goal
  unsigned long long total = 0, all, before = 0;
  for (int t = tid; t < c.tiles; t += kThreads) total += tiles[t];
  scan(total, sh.parts, turn, all);
  total = all;
  const float u = fminf(fmaxf(c.a.uniform[r], 0.f), 0x1.fffffep-1f);
  double goal = static_cast<double>(u) * static_cast<double>(total);
  for (int t0 = 0;; t0 += kThreads) {
    const unsigned long long s = t0 + tid < c.tiles ? tiles[t0 + tid] : 0;
    const unsigned long long upto = before + scan(s, sh.parts, turn, all);
    if (s != 0 && static_cast<double>(upto) > goal && static_cast<double>(upto - s) <= goal) {
      sh.at = t0 + tid;
      sh.wide = upto - s;
    }
    before += all;
    if (static_cast<double>(before) > goal || t0 + kThreads >= c.tiles) break;
  }
  __syncthreads();
  // and the token in it
  static_assert(kTile == kThreads, "a token a thread");
  const int tile = sh.at, i = tile * kTile + tid;
  const float own_v = i < vocab ? get(x + i) : -__builtin_inff();
  before = sh.wide;
  double chance = 0.0;
  if (i < vocab && c.a.prob) chance = row.weight(row.seen(own_v)) / static_cast<double>(total);
  if constexpr (TILES) {  // in the tile's own weights
    const double own = static_cast<double>(c.w.sums[static_cast<int64_t>(r) * c.tiles + tile]);
    // (below own, whatever the product is rounded to: own can be 2^60, where own - 1 is own)
    goal = fmin((goal - static_cast<double>(before)) * (own / static_cast<double>(tiles[tile])), own * (1.0 - 0x1p-53));
    before = 0;
    row.against(value_of(c.w.ends[static_cast<int64_t>(r) * c.tiles + tile].x));
  }
  const unsigned long long k = i < vocab ? kept(row.seen(own_v), i) : 0;
  const unsigned long long upto = before + scan(k, sh.parts, turn, all);
  if (k != 0 && static_cast<double>(upto) > goal && static_cast<double>(upto - k) <= goal) answer(i, static_cast<float>(chance));
}

// ------------------------------------------------------------------------------ launch

struct Sizes {
  int tiles;
  size_t ends, sums, weights, counts, listed, plans, list, bytes;
};
Sizes sizes(int32_t rows, int32_t vocab) {
  Sizes z{};
  z.tiles = (vocab + kTile - 1) / kTile;
  size_t at = 0;
  const auto room = [&](size_t& from, size_t bytes) {
    from = at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
  };
  const size_t r = rows;
  room(z.ends, r * z.tiles * sizeof(uint2));
  room(z.sums, r * z.tiles * 8);
  room(z.weights, r * kBins * 8);
  room(z.counts, r * kBins * 4);
  room(z.listed, r * 4);
  room(z.plans, r * sizeof(Plan));
  room(z.list, r * kList * 4);
  z.bytes = at;
  return z;
}

template <typename T>
hipError_t launch_t(Call c, hipStream_t s) {
  const int64_t most = (int64_t{1} << 31) / kThreads / c.groups;  // rows of a launch
  const int rows = c.a.rows;
  const size_t lds = static_cast<size_t>(c.tiles) * 8;
  const bool borders = c.a.top_k || c.a.top_p, own = !borders && !c.a.min_p;
  for (int64_t f = 0; f < rows; f += most) {
    c.first = static_cast<int>(f);
    const unsigned n = static_cast<unsigned>(rows - f < most ? rows - f : most);
    if (own) {
      sample_tiles_kernel<T><<<n * c.groups, kThreads, 0, s>>>(c);
      sample_choose_kernel<T, true><<<n, kThreads, lds, s>>>(c);
    } else {
      sample_extremes_kernel<T><<<n * c.groups, kThreads, 0, s>>>(c);
      sample_weigh_kernel<T><<<n * c.groups, kThreads, 0, s>>>(c);
      if (borders) sample_gather_kernel<T><<<n * c.groups, kThreads, 0, s>>>(c);
      sample_choose_kernel<T, false><<<n, kThreads, lds, s>>>(c);
    }
    if (const hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t sample_workspace_bytes(int32_t rows, int32_t vocab) { return sizes(rows, vocab).bytes; }

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  const Sizes z = sizes(a.rows, a.vocab);
  char* ws = static_cast<char*>(a.workspace);
  const bool filters = a.top_k || a.top_p;
  Call c{};
  c.a = a;
  c.w = Space{reinterpret_cast<uint2*>(ws + z.ends),
              reinterpret_cast<unsigned long long*>(ws + z.sums),
              reinterpret_cast<unsigned long long*>(ws + z.weights),
              filters ? reinterpret_cast<uint32_t*>(ws + z.counts) : nullptr,
              reinterpret_cast<uint32_t*>(ws + z.listed),
              reinterpret_cast<Plan*>(ws + z.plans),
              reinterpret_cast<uint32_t*>(ws + z.list)};
  c.tiles = z.tiles;
  int bits = 0;
  while ((1 << bits) < a.vocab) ++bits;
  c.shift = 62 - bits < 51 ? 62 - bits : 51;
  // about three workgroups a CU in the passes over all tokens (64 rows of 99991 with filters, the kernels' sum: 576 workgroups
  // 43.4 us, 768 40.1, 832 42.2, 1600 48.5)
  const int blocks = (z.tiles + kWaves - 1) / kWaves;
  const int want = (768 + a.rows - 1) / a.rows;
  c.groups = want < blocks ? want : blocks;
  return a.bf16 ? launch_t<uint16_t>(c, s) : launch_t<float>(c, s);
}

}  // namespace gdn
