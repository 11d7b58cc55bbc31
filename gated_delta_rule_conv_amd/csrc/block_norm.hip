// The norms around a block of a residual stream, gfx950 (include/gdn.h, gdn_block_norm):
//   a = N(x) post_w + post_b,  h = r + scale act(gate) a,  y = N(h) pre_w + pre_b.
//
// Bound by HBM: x, r and the gate are read once, h and y written once. A row lives in the registers of W waves
// (lane c of the row's 64 W: values [8 (c + 64 W t), + 8), t < V), so both norms are sums over registers
// and h goes from its sum to its norm unrounded.

#include "conv_taps.h"
#include "device_common.h"
#include "launch.h"
#include "norm_values.h"

#include "../../include/gdn.h"

namespace gdn {
namespace {

// values [k, k + 8) of a row of n
__device__ __forceinline__ void load8(const void* p, int bf16, int64_t off, int k, int n, float (&v)[8]) {
  const f32x4 lo = load_any(p, bf16, off, k, n), hi = load_any(p, bf16, off, k + 4, n);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = lo[e];
    v[4 + e] = hi[e];
  }
}

__device__ __forceinline__ void store8(void* p, int bf16, int64_t off, int k, int n, const float (&v)[8]) {
  const f32x4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
  if (bf16) {
    store4u(static_cast<uint16_t*>(p) + off, k, n, lo);
    store4u(static_cast<uint16_t*>(p) + off, k + 4, n, hi);
  } else {
    store4u(static_cast<float*>(p) + off, k, n, lo);
    store4u(static_cast<float*>(p) + off, k + 4, n, hi);
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
    const int wave = threadIdx.x / kWave;
    turn ^= 1;  // (the readers of the last turn's values need not be done)
    if (threadIdx.x % kWave == 0) part[turn][wave] = v;
    __syncthreads();
    float r = part[turn][0];
#pragma unroll
    for (int w = 1; w < W; ++w) r = join(r, part[turn][w]);
    return r;
  }
};

// v -> (v - mean) rs over a row: the root mean square's inverse, or, centered, the standard deviation's.
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

template <int W, int V>
__global__ __launch_bounds__((W < 4 ? 4 : W) * kWave) void block_norm_kernel(BlockNormArgs a) {
  __shared__ float part[2][16];
  Gather<W> gather{part};
  constexpr int ROWS = W < 4 ? 4 / W : 1;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x / (W * kWave) : 0);
  if (row >= a.rows) return;  // (W = 1: no barrier follows)
  const int c = threadIdx.x % (W * kWave), n = a.width;
  const auto at = [&](int t) { return 8 * (c + W * kWave * t); };
  float v[V][8];
#pragma unroll
  for (int t = 0; t < V; ++t) load8(a.x, a.x_bf16, row * a.x_stride, at(t), n, v[t]);
  const auto apply = [&](const void* w, const void* b) {
    if (w) {
#pragma unroll
      for (int t = 0; t < V; ++t) {
        float p[8];
        load8(w, a.param_bf16, 0, at(t), n, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[t][e] *= p[e];
      }
    }
    if (b) {
#pragma unroll
      for (int t = 0; t < V; ++t) {
        float p[8];
        load8(b, a.param_bf16, 0, at(t), n, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[t][e] += p[e];
      }
    }
  };
  if (a.post) {
    normalise<W, V>(v, a, c, gather);
    apply(a.post_weight, a.post_bias);
  }
  if (a.gate) {
#pragma unroll
    for (int t = 0; t < V; ++t) {
      float z[8];
      load8(a.gate, a.gate_bf16, row * a.gate_stride, at(t), n, z);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[t][e] *= a.activation == GDN_ACT_NONE ? z[e] : a.activation == GDN_ACT_SILU ? silu(z[e]) : sigmoid(z[e]);
    }
  }
#pragma unroll
  for (int t = 0; t < V; ++t) {
    float r[8] = {};
    if (a.residual) load8(a.residual, a.residual_bf16, row * a.residual_stride, at(t), n, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[t][e] = at(t) + e < n ? fmaf(a.scale, v[t][e], r[e]) : 0.f;
    if (a.h) store8(a.h, a.residual_bf16, row * a.h_stride, at(t), n, v[t]);
  }
  if (!a.y) return;
  normalise<W, V>(v, a, c, gather);
  apply(a.pre_weight, a.pre_bias);
#pragma unroll
  for (int t = 0; t < V; ++t) store8(a.y, a.y_bf16, row * a.y_stride, at(t), n, v[t]);
}

template <int W, int V>
hipError_t launch_v(const BlockNormArgs& a, hipStream_t s) {
  constexpr int rows = W < 4 ? 4 / W : 1;
  block_norm_kernel<W, V><<<static_cast<unsigned>((a.rows + rows - 1) / rows), (W < 4 ? 4 : W) * kWave, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

namespace {
hipError_t launch_rows(const BlockNormArgs& a, hipStream_t s) {
  if (a.width <= 512) return launch_v<1, 1>(a, s);
  if (a.width <= 1024) return launch_v<1, 2>(a, s);
  if (a.width <= 2048) return launch_v<4, 1>(a, s);
  if (a.width <= 4096) return launch_v<4, 2>(a, s);
  if (a.width <= 8192) return launch_v<4, 4>(a, s);
  if (a.width <= 16384) return launch_v<16, 2>(a, s);
  return launch_v<16, 4>(a, s);
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
    const hipError_t e = launch_rows(a, s);
    if (e != hipSuccess || args.rows - r <= most) return e;
    r += most;
  }
}

}  // namespace gdn
