// One token a row of logits from a given random number, gfx950 (include/gdn.h, gdn_sample).
//
// Weights are whole numbers: w = round(2^S e^((x - m) / T)), the exponential in 64 bits, S = 62 minus
// the bits of the vocabulary's size (44 for 2^18 tokens). Their sums are then exact in any order, so a row's
// token depends on nothing but the row, and a border (top_p's, or the random number's) is met within 2^-S of
// the largest weight a token. Values are ordered by a key that sorts as an unsigned number, so a filter's
// border is found by counting (top_k) or weighing (top_p) the 2048 values of the key's leading 11 bits, then
// the next 11 inside that bin, then the last 10; among equal values the lower index comes first.

#include "device_common.h"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr uint32_t kLowest = 0x007FFFFFu;  // key_of(-infinity)
constexpr int kTile = 4 * kThreads;         // tokens whose weights are summed together
constexpr int kMaxTiles = (1 << 24) / kTile;

template <typename T>
__device__ __forceinline__ uint32_t key_of(T raw) {
  float x;
  if constexpr (sizeof(T) == 2) x = bf16_to_f32(raw);
  else x = raw;
  if (!(x == x)) return kLowest;  // a NaN is a token that cannot come
  x += 0.0f;                      // (-0 is 0)
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// 2^t for t <= 0: the series of e^(f ln 2) for the part of t past its nearest whole number, |f| <= 1/2 (the first
// term left out is under 2^-52), times a power of two.
__device__ __forceinline__ double power_of_two(double t) {
  t = t < -1100.0 ? -1100.0 : t;
  const double n = rint(t), f = (t - n) * 0.693147180559945309417;
  double s = 1.0 / 479001600.0;
  s = fma(s, f, 1.0 / 39916800.0);
  s = fma(s, f, 1.0 / 3628800.0);
  s = fma(s, f, 1.0 / 362880.0);
  s = fma(s, f, 1.0 / 40320.0);
  s = fma(s, f, 1.0 / 5040.0);
  s = fma(s, f, 1.0 / 720.0);
  s = fma(s, f, 1.0 / 120.0);
  s = fma(s, f, 1.0 / 24.0);
  s = fma(s, f, 1.0 / 6.0);
  s = fma(s, f, 0.5);
  s = fma(s, f, 1.0);
  s = fma(s, f, 1.0);
  return ldexp(s, static_cast<int>(n));
}

struct Row {
  float most;       // the largest value
  double per;       // log2(e) / T
  double least;     // min_p, at most 1
  int shift;        // S
  // e^((x - most) / T), of the largest value 1
  __device__ __forceinline__ double weight(uint32_t key) const {
    if (key == kLowest) return 0.0;
    const float x = value_of(key);
    if (x == most) return 1.0;
    return power_of_two((static_cast<double>(x) - static_cast<double>(most)) * per);
  }
  __device__ __forceinline__ uint64_t whole(double w) const { return static_cast<uint64_t>(rint(ldexp(w, shift))); }
};


struct Shared {
  uint32_t count[2048];
  unsigned long long weight[2048];
  unsigned long long tile[kMaxTiles];
  unsigned long long part[kThreads / kWave];
  uint32_t most;
  uint32_t prefix;
  uint32_t at;
  unsigned long long before;
  uint32_t found;
};

// Where a filter's order ends: every key above `key`, and of the equal ones the first `equal` by index.
struct Border {
  uint32_t key;
  uint32_t equal;
};

// The border of the first `want` tokens (BY_COUNT), or of those before which less than `target` of weight lies, among the tokens
// up to `limit`'s border. `total` gets the weight up to the border.
template <typename T, bool BY_COUNT>
__device__ Border find(const T* x, int vocab, const Row& row, const Border& limit, uint32_t want, double target, Shared& sh) {
  const int tid = threadIdx.x;
  uint32_t prefix = 0;         // the leading bits found so far
  unsigned long long before = 0;  // count or weight of the keys above them
  int left = 32;
  for (int level = 0; level < 3; ++level) {
    const int bits = level == 2 ? 10 : 11, bins = 1 << bits, low = left - bits;
    for (int b = tid; b < bins; b += kThreads) {
      sh.count[b] = 0;
      sh.weight[b] = 0;
    }
    __syncthreads();
    for (int i = tid; i < vocab; i += kThreads) {
      const uint32_t key = key_of(x[i]);
      if (key < limit.key || (level > 0 && (key >> left) != prefix)) continue;
      const uint32_t b = (key >> low) & (bins - 1);
      atomicAdd(&sh.count[b], 1u);
      if (!BY_COUNT && key > limit.key) atomicAdd(&sh.weight[b], static_cast<unsigned long long>(row.whole(row.weight(key))));
    }
    __syncthreads();
    if (tid == 0) {
      if (!BY_COUNT && limit.key != 0 && (level == 0 || (limit.key >> left) == prefix)) {
        const uint32_t b = (limit.key >> low) & (bins - 1);
        sh.weight[b] += limit.equal * static_cast<unsigned long long>(row.whole(row.weight(limit.key)));
      }
      int at = -1;
      unsigned long long sum = before, sum_at = before;
      for (int b = bins - 1; b >= 0; --b) {
        if (sh.count[b] == 0) continue;
        if (at >= 0 && (BY_COUNT ? sum >= want : static_cast<double>(sum) >= target)) break;
        at = b;
        sum_at = sum;
        sum += BY_COUNT ? sh.count[b] : sh.weight[b];
      }
      sh.at = at;
      sh.before = sum_at;
      sh.found = sh.count[at];
    }
    __syncthreads();
    prefix = level == 0 ? sh.at : (prefix << bits) | sh.at;
    before = sh.before;
    left = low;
    __syncthreads();
  }
  Border out{prefix, sh.found};
  if (out.key == limit.key) out.equal = min(out.equal, limit.equal);
  if (BY_COUNT) {
    out.equal = min(out.equal, static_cast<uint32_t>(want - before));
  } else {
    const unsigned long long w = row.whole(row.weight(out.key));
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

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs a, int shift) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), r = blockIdx.x, vocab = a.vocab;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  if (tid == 0) sh.most = 0;
  __syncthreads();
  uint32_t most = 0;
  for (int i = tid; i < vocab; i += kThreads) most = max(most, key_of(x[i]));
  atomicMax(&sh.most, most);
  __syncthreads();
  most = sh.most;
  if (most == kLowest) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.prob) a.prob[r] = 0.f;
    }
    return;
  }
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  if (tid == 0) sh.at = vocab;
  __syncthreads();
  if (!(t > 0.f)) {
    for (int i = tid; i < vocab; i += kThreads)
      if (key_of(x[i]) == most) {
        atomicMin(&sh.at, static_cast<uint32_t>(i));
        break;
      }
    __syncthreads();
    if (tid == 0) {
      a.tokens[r] = sh.at;
      if (a.prob) a.prob[r] = 1.f;
    }
    return;
  }
  Row row{value_of(most), 1.44269504088896340736 / static_cast<double>(t), 0.0, shift};
  const float least = a.min_p ? a.min_p[r] : 0.f;
  row.least = least > 0.f ? (least < 1.f ? least : 1.0) : 0.0;
  const int32_t k = a.top_k ? a.top_k[r] : 0;
  const float p = a.top_p ? a.top_p[r] : 1.f;
  Border border{0, static_cast<uint32_t>(vocab)};
  if (k > 0 && k < vocab) border = find<T, true>(x, vocab, row, border, k, 0.0, sh);
  // the index behind which equal keys are out
  const auto cut_of = [&](const Border& b) {
    __syncthreads();
    if (tid == 0) sh.at = 0xFFFFFFFFu;
    uint32_t seen = 0;
    for (int i0 = 0; i0 < vocab && b.key != 0; i0 += kThreads) {
      const int i = i0 + tid;
      const bool eq = i < vocab && key_of(x[i]) == b.key;
      const uint64_t mask = __ballot(eq);
      __syncthreads();
      if (lane == 0) sh.part[tid / kWave] = __popcll(mask);
      __syncthreads();
      uint32_t mine = seen + __popcll(mask & ((1ull << lane) - 1));
      for (int w = 0; w < kThreads / kWave; ++w) {
        if (w < tid / kWave) mine += sh.part[w];
        seen += sh.part[w];
      }
      if (eq && mine + 1 == b.equal) sh.at = i;
      if (seen >= b.equal) break;
    }
    __syncthreads();
    return sh.at;
  };
  uint32_t cut = cut_of(border);
  const auto weight = [&](int i, bool floor) -> uint64_t {
    const uint32_t key = key_of(x[i]);
    if (key < border.key || (key == border.key && static_cast<uint32_t>(i) > cut)) return 0;
    const double w = row.weight(key);
    return floor && w < row.least ? 0 : row.whole(w);
  };
  const auto sum_all = [&](bool floor) {
    const int tiles = (vocab + kTile - 1) / kTile;
    __syncthreads();
    for (int i = tid; i < tiles; i += kThreads) sh.tile[i] = 0;
    __syncthreads();
    for (int n = 0; n < tiles; ++n) {
      unsigned long long s = 0;
      for (int i = n * kTile + tid; i < min(vocab, (n + 1) * kTile); i += kThreads) s += weight(i, floor);
#pragma unroll
      for (int m = 1; m < kWave; m *= 2) s += __shfl_xor(s, m);
      if (lane == 0) atomicAdd(&sh.tile[n], s);
    }
    __syncthreads();
    unsigned long long s = 0;
    for (int n = 0; n < tiles; ++n) s += sh.tile[n];
    return s;
  };
  if (p < 1.f) {
    const double target = static_cast<double>(p) * static_cast<double>(sum_all(false));
    __syncthreads();
    border = find<T, false>(x, vocab, row, border, 0, target, sh);
    cut = cut_of(border);
  }
  const unsigned long long total = sum_all(true);
  const float u = fminf(fmaxf(a.uniform[r], 0.f), 0x1.fffffep-1f);
  const double goal = static_cast<double>(u) * static_cast<double>(total);
  int n = 0;
  unsigned long long before = 0;
  while (static_cast<double>(before + sh.tile[n]) <= goal) before += sh.tile[n++];
  // the tile's tokens, 1024 at a time
  for (int i0 = n * kTile;; i0 += kThreads) {
    const int i = i0 + tid;
    const unsigned long long w = i < vocab ? weight(i, true) : 0;
    unsigned long long s = w;
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
      const unsigned long long o = __shfl_up(s, m);
      if (lane >= m) s += o;
    }
    __syncthreads();
    if (lane == kWave - 1) sh.part[tid / kWave] = s;
    __syncthreads();
    unsigned long long all = 0;
    s += before;
    for (int v = 0; v < kThreads / kWave; ++v) {
      if (v < tid / kWave) s += sh.part[v];
      all += sh.part[v];
    }
    if (w != 0 && static_cast<double>(s) > goal && static_cast<double>(s - w) <= goal) {
      a.tokens[r] = i;
      if (a.prob) a.prob[r] = static_cast<float>(row.weight(key_of(x[i])) / ldexp(static_cast<double>(total), -shift));
    }
    before += all;
    if (static_cast<double>(before) > goal || i0 + kThreads >= vocab) break;
  }
}

}  // namespace

size_t sample_workspace_bytes(int32_t, int32_t) { return 0; }

hipError_t launch_sample(const SampleArgs& a, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < a.vocab) ++bits;
  const int shift = 62 - bits < 52 ? 62 - bits : 52;
  if (a.bf16) sample_kernel<uint16_t><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a, shift);
  else sample_kernel<float><<<static_cast<unsigned>(a.rows), kThreads, 0, s>>>(a, shift);
  return hipGetLastError();
}

}  // namespace gdn
