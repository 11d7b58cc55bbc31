// The norms around a block of a residual stream, gfx950 (include/gdn.h, gdn_block_norm):
//   a = N(x) post_w + post_b,  h = r + scale act(gate) a,  y = N(h) pre_w + pre_b.
//
// Bound by HBM: x, r and the gate are read once, h and y written once. A row lives in the registers of W waves
// (lane c of the row's 64 W: values [8 (c + 64 W t), + 8), t < V), so both norms are sums over registers
// and h goes from its sum to its norm unrounded. x, r and the gate are loaded as they come before anything is computed, which is
// why their types are compiled in (chosen at run time the loads waited for each other: 15717 rows of 4096 242 us against 158, 5.7
// TB/s); the parameters come from L2 while the sums run. 64 rows: 4.5 us, three memory round trips and two joined sums.

#include "conv_taps.h"
#include "device_common.h"
#include "launch.h"
#include "norm_values.h"

#include "../../include/gdn.h"

namespace gdn {
namespace {

typedef uint32_t uu32x4 __attribute__((ext_vector_type(4), aligned(2)));
struct None {};

// 8 values as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  uu32x4 r;
  __device__ __forceinline__ void load(const uint16_t* p) { r = *reinterpret_cast<const uu32x4*>(p); }
  __device__ __forceinline__ void set(int e, uint16_t v) {
    const uint32_t old = r[e / 2];
    r[e / 2] = e % 2 ? (old & 0xFFFFu) | static_cast<uint32_t>(v) << 16 : (old & 0xFFFF0000u) | v;
  }
  __device__ __forceinline__ void clear() { r = uu32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float operator[](int e) const {
    return __uint_as_float(e % 2 ? r[e / 2] & 0xFFFF0000u : r[e / 2] << 16);
  }
};
template <>
struct Raw8<float> {
  uf32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const uf32x4*>(p);
    b = *reinterpret_cast<const uf32x4*>(p + 4);
  }
  __device__ __forceinline__ void set(int e, float v) {
    if (e < 4) a[e] = v;
    else b[e - 4] = v;
  }
  __device__ __forceinline__ void clear() { a = b = uf32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ float operator[](int e) const { return e < 4 ? a[e] : b[e - 4]; }
};
template <>
struct Raw8<None> {
  __device__ __forceinline__ float operator[](int) const { return 1.f; }
};

// values [k, k + 8) of a row of n. EIGHTS: 8 divides n, so that a lane has all of them or (k >= n) none: it reads the row's
// first ones then, and what it forms of them is dropped.
template <bool EIGHTS, typename T>
__device__ __forceinline__ void load8(Raw8<T>& to, const void* row, int k, int n) {
  if constexpr (sizeof(Raw8<T>) >= 16) {
    const T* p = static_cast<const T*>(row);
    if constexpr (EIGHTS) {
      to.load(p + (k < n ? k : 0));
    } else if (k + 8 <= n) {
      to.load(p + k);
    } else {
      to.clear();
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < n) to.set(e, p[k + e]);
    }
  }
}

template <bool EIGHTS, typename T>
__device__ __forceinline__ void store8(T* p, int k, int n, const float (&v)[8]) {
  if (EIGHTS ? k < n : k + 8 <= n) {
    if constexpr (sizeof(T) == 2) {
      uu32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = static_cast<uint32_t>(to_bf16(v[2 * e])) | static_cast<uint32_t>(to_bf16(v[2 * e + 1])) << 16;
      *reinterpret_cast<uu32x4*>(p + k) = r;
    } else {
      *reinterpret_cast<uf32x4*>(p + k) = uf32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<uf32x4*>(p + k + 4) = uf32x4{v[4], v[5], v[6], v[7]};
    }
  } else if constexpr (!EIGHTS) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < n) put(p + k + e, v[e]);
  }
}

__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f));
}

// Over the W waves of a row, in a fixed order.
template <int W>
struct Gather {
  float (&part)[2][16];
  int turn = 0;
  template <typename F>
  __device__ __forceinline__ float operator()(float v, F join) {
    if constexpr (W == 1) return v;
    turn ^= 1;  // (the readers of the last turn's values need not be done)
    if (threadIdx.x % kWave == 0) part[turn][threadIdx.x / kWave] = v;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");  // (loads stay in flight)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    float r = part[turn][0];
#pragma unroll
    for (int w = 1; w < W; ++w) r = join(r, part[turn][w]);
    return r;
  }
};

// v -> (v - mean) rs over a row: the root mean square's inverse, or, centered, the standard deviation's. v is 0 past the row's end.
template <int W, int V>
__device__ __forceinline__ void normalise(float (&v)[V][8], const BlockNormArgs& a, int c, Gather<W>& gather) {
  const auto add = [](float x, float y) { return x + y; };
  const float per = 1.0f / static_cast<float>(a.width);
  float mean = 0.f;
  const auto mean_square = [&]() {
    if (a.centered) {
      float s = 0.f;
#pragma unroll
      for (int t = 0; t < V; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[t][e];
      mean = gather(lanes_sum<kWave>(s), add) * per;
    }
    float q = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = !a.centered || 8 * (c + W * kWave * t) + e < a.width ? v[t][e] - mean : 0.f;
        q = fmaf(d, d, q);
      }
    return gather(lanes_sum<kWave>(q), add) * per;
  };
  const float ms = mean_square() + a.eps;
  float rs = __builtin_amdgcn_rsqf(ms);
  if (!in_range(ms)) {  // (the row agrees)
    float most = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(v[t][e]));
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
    most = gather(most, [](float x, float y) { return fmaxf(x, y); });
    const int sh = range_shift(most, a.eps);
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[t][e] = ldexpf(v[t][e], sh);
    rs = 1.0f / sqrtf(mean_square() + ldexpf(a.eps, 2 * sh));
  }
#pragma unroll
  for (int t = 0; t < V; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[t][e] = (v[t][e] - mean) * rs;
}

template <typename TX, typename TR, typename TZ, int W, int V, bool EIGHTS>
__global__ __launch_bounds__((W < 4 ? 4 : W) * kWave) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float part[2][16];
  static_assert(W == 1 || W >= 4, "whole workgroups, or waves on their own");
  Gather<W> gather{part};
  constexpr int ROWS = W < 4 ? 4 / W : 1;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x / (W * kWave) : 0);
  if (row >= a.rows) return;  // (W = 1: no barrier follows)
  const int c = threadIdx.x % (W * kWave), n = a.width;
  const auto at = [&](int t) { return 8 * (c + W * kWave * t); };
  const auto row_of = [&](const auto* p, int64_t stride) { return p + row * stride; };
  Raw8<TX> x[V];
  Raw8<TZ> z[V];
  Raw8<TR> r[V];
#pragma unroll
  for (int t = 0; t < V; ++t) load8<EIGHTS>(x[t], row_of(static_cast<const TX*>(a.x), a.x_stride), at(t), n);
  if constexpr (sizeof(TZ) > 1) {
#pragma unroll
    for (int t = 0; t < V; ++t) load8<EIGHTS>(z[t], row_of(static_cast<const TZ*>(a.gate), a.gate_stride), at(t), n);
  }
  if (a.residual) {
#pragma unroll
    for (int t = 0; t < V; ++t) load8<EIGHTS>(r[t], row_of(static_cast<const TR*>(a.residual), a.residual_stride), at(t), n);
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) r[t].clear();
  }
  float v[V][8];
#pragma unroll
  for (int t = 0; t < V; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[t][e] = !EIGHTS || at(t) < n ? x[t][e] : 0.f;
  // v = v w + b, where they are given
  const auto affine = [&](const void* w, const void* b) {
    const auto with = [&](auto zero, const void* p, auto join) {
      using T = decltype(zero);
#pragma unroll
      for (int t = 0; t < V; ++t) {
        Raw8<T> q;
        load8<EIGHTS>(q, p, at(t), n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[t][e] = join(v[t][e], q[e]);
      }
    };
    const auto times = [](float p, float q) { return p * q; };
    const auto plus = [](float p, float q) { return p + q; };
    if (w) a.param_bf16 ? with(uint16_t{}, w, times) : with(float{}, w, times);
    if (b) a.param_bf16 ? with(uint16_t{}, b, plus) : with(float{}, b, plus);
  };
  if (a.post) {
    normalise<W, V>(v, a, c, gather);
    affine(a.post_weight, a.post_bias);
  }
  if constexpr (sizeof(TZ) > 1) {
    const auto gate = [&](auto act) {
#pragma unroll
      for (int t = 0; t < V; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[t][e] *= act(z[t][e]);
    };
    if (a.activation == GDN_ACT_NONE) gate([](float p) { return p; });
    else if (a.activation == GDN_ACT_SILU) gate([](float p) { return silu(p); });
    else gate([](float p) { return sigmoid(p); });
  }
#pragma unroll
  for (int t = 0; t < V; ++t) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[t][e] = at(t) + (EIGHTS ? 0 : e) < n ? fmaf(a.scale, v[t][e], r[t][e]) : 0.f;
    if (a.h) store8<EIGHTS>(static_cast<TR*>(a.h) + row * a.h_stride, at(t), n, v[t]);
  }
  if (!a.y) return;
  normalise<W, V>(v, a, c, gather);
  affine(a.pre_weight, a.pre_bias);
#pragma unroll
  for (int t = 0; t < V; ++t) {
    if (a.y_bf16) store8<EIGHTS>(static_cast<uint16_t*>(a.y) + row * a.y_stride, at(t), n, v[t]);
    else store8<EIGHTS>(static_cast<float*>(a.y) + row * a.y_stride, at(t), n, v[t]);
  }
}

template <typename TX, typename TR, typename TZ, int W, int V, bool EIGHTS>
hipError_t launch_v(const BlockNormArgs& a, hipStream_t s) {
  constexpr int rows = W < 4 ? 4 / W : 1;
  block_norm_kernel<TX, TR, TZ, W, V, EIGHTS>
      <<<static_cast<unsigned>((a.rows + rows - 1) / rows), (W < 4 ? 4 : W) * kWave, 0, s>>>(a);
  return hipGetLastError();
}

// Waves a row, and groups of 8 values a lane: of these shapes the one with the fewest idle lanes, then the most waves (64 Mi bf16 values of x, residual, gate,
// h and y, TB/s: width 1024 with 4 waves 4.9, one wave with two groups 5.6; 2048 with 4 waves 5.7, with two groups 5.4;
// 4104 with 16 waves 4.5, 8 with two groups 4.8; 16384 with two groups 4.8, four 3.9). With four groups 16 waves have 128 registers
// each, which suffices where 8 divides the width for bf16 throughout, and for one of x and residual in fp32 without a gate; the rest spills
// (16 to 276 bytes a lane): 32768 wide 5.0 TB/s in bf16, 4.0 in fp32, 32767 wide 2.7 and 3.5.
template <typename TX, typename TR, typename TZ, bool EIGHTS>
hipError_t launch_w(const BlockNormArgs& a, hipStream_t s) {
  if (a.width <= 512) return launch_v<TX, TR, TZ, 1, 1, EIGHTS>(a, s);
  if (a.width <= 1024) return launch_v<TX, TR, TZ, 1, 2, EIGHTS>(a, s);
  if (a.width <= 2048) return launch_v<TX, TR, TZ, 4, 1, EIGHTS>(a, s);
  if (a.width <= 4096) return launch_v<TX, TR, TZ, 8, 1, EIGHTS>(a, s);
  if (a.width <= 8192) return launch_v<TX, TR, TZ, 8, 2, EIGHTS>(a, s);
  if (a.width <= 16384) return launch_v<TX, TR, TZ, 16, 2, EIGHTS>(a, s);
  return launch_v<TX, TR, TZ, 16, 4, EIGHTS>(a, s);
}

template <typename TX, typename TR, typename TZ>
hipError_t launch_t(const BlockNormArgs& a, hipStream_t s) {
  return a.width % 8 == 0 ? launch_w<TX, TR, TZ, true>(a, s) : launch_w<TX, TR, TZ, false>(a, s);
}

template <typename TX, typename TR>
hipError_t launch_z(const BlockNormArgs& a, hipStream_t s) {
  if (!a.gate) return launch_t<TX, TR, None>(a, s);
  return a.gate_bf16 ? launch_t<TX, TR, uint16_t>(a, s) : launch_t<TX, TR, float>(a, s);
}

}  // namespace

// A launch holds fewer than 2^32 threads: calls of more than 2^21 rows (1024 threads each at most) go in pieces.
hipError_t launch_block_norm(const BlockNormArgs& args, hipStream_t s) {
  constexpr int32_t most = 1 << 21;
  for (int32_t r = 0;;) {
    BlockNormArgs a = args;
    a.rows = args.rows - r < most ? args.rows - r : most;
    const auto at = [r](const void* p, int bf16, int64_t stride) {
      return p ? static_cast<const char*>(p) + r * stride * (bf16 ? 2 : 4) : nullptr;
    };
    a.x = at(args.x, a.x_bf16, a.x_stride);
    a.residual = at(args.residual, a.residual_bf16, a.residual_stride);
    a.gate = at(args.gate, a.gate_bf16, a.gate_stride);
    a.h = const_cast<char*>(at(args.h, a.residual_bf16, a.h_stride));
    a.y = const_cast<char*>(at(args.y, a.y_bf16, a.y_stride));
    const hipError_t e = a.x_bf16 ? (a.residual_bf16 ? launch_z<uint16_t, uint16_t>(a, s) : launch_z<uint16_t, float>(a, s))
                                  : (a.residual_bf16 ? launch_z<float, uint16_t>(a, s) : launch_z<float, float>(a, s));
    if (e != hipSuccess || args.rows - r <= most) return e;
    r += most;
  }
}

}  // namespace gdn
