// The norm of every group of channels of every token, with its activation and gate, gfx950
// (include/gdn.h, gdn_group_norm): n = x / sqrt(mean x^2 + eps), or the same of x - mean(x);
// y = (n w + b) act(gate).
//
// Bound by HBM, with the vector units close behind: x, gate and y move once (8 bytes a value for fp32 x and
// bf16 gate and y: 515 MB of a 15717-token, 32-head, d = 128 layer in 95 us, 5.4 TB/s), and a value takes
// about 12 VALU operations besides the exponential and the reciprocal of SiLU, which cost four times one;
// so the divisions by the group count and size are products with numbers the host prepared (the mean is then good to
// an ulp), and the root is the hardware's reciprocal square root (an ulp as well). A group lives in the registers of LPG adjacent lanes, each
// holding V vectors of 4 consecutive values (lane c: values 4 (c + LPG t), t < V), so the mean
// and the sum of squares are one pass over memory and two over registers, in fp32; sums over lanes
// are fixed butterflies. Rows and groups may start at any multiple of the element: gfx950's vector
// loads take any address, so no size or stride needs a scalar form, except for a group's last
// vector when 4 does not divide its size.

#include "conv_taps.h"
#include "device_common.h"
#include "launch.h"

namespace gdn {
namespace {

constexpr int kNormWaves = 4;

// 4 values as fp32 from an address aligned to the element only
typedef float uf32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t uu16x4 __attribute__((ext_vector_type(4), aligned(2)));

template <typename T>
__device__ __forceinline__ float get(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}

// (the hardware conversion: nearest even, and a NaN of any payload stays one)
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = to_bf16(v);
  else *p = v;
}

// values [k, k + 4) of a group of `size`, zeros past its end
template <typename T>
__device__ __forceinline__ f32x4 load4u(const T* p, int k, int size) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (k + 3 < size) {
    if constexpr (sizeof(T) == 2) {
      const uu16x4 r = *reinterpret_cast<const uu16x4*>(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = bf16_to_f32(r[e]);
    } else {
      const uf32x4 r = *reinterpret_cast<const uf32x4*>(p + k);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = r[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (k + e < size) v[e] = get(p + k + e);
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store4u(T* p, int k, int size, const f32x4& v) {
  if (k + 3 < size) {
    if constexpr (sizeof(T) == 2) {
      uu16x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = to_bf16(v[e]);
      *reinterpret_cast<uu16x4*>(p + k) = r;
    } else {
      uf32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = v[e];
      *reinterpret_cast<uf32x4*>(p + k) = r;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 3; ++e)
      if (k + e < size) put(p + k + e, v[e]);
  }
}

__device__ __forceinline__ f32x4 load_any(const void* p, int bf16, int64_t off, int k, int size) {
  return bf16 ? load4u(static_cast<const uint16_t*>(p) + off, k, size)
              : load4u(static_cast<const float*>(p) + off, k, size);
}

// a lane's V vectors of a group
template <int LPG, int V>
__device__ __forceinline__ void load_all(const void* p, int bf16, int64_t off, int c, int size, f32x4 (&v)[V]) {
  if (bf16) {
#pragma unroll
    for (int t = 0; t < V; ++t) v[t] = load4u(static_cast<const uint16_t*>(p) + off, 4 * (c + LPG * t), size);
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) v[t] = load4u(static_cast<const float*>(p) + off, 4 * (c + LPG * t), size);
  }
}

// Sum over aligned groups of L lanes, the last two steps by gfx950's swaps of lane rows.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  v = group_sum<(L < 16 ? L : 16)>(v);
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// Squares leave the fp32 range long before values do. Where the mean square is not a number well inside it
// (overflow, underflow, an infinity in the group), the group is taken again times 2^range_shift, which puts the
// larger of its largest magnitude and sqrt(eps) near 1. Only such groups pay: 15717 x 32 x 128 fp32 values take 94 us
// with the test and without.
__device__ __forceinline__ bool in_range(float ms) { return ms > 0x1p-100f && ms < __builtin_inff(); }
__device__ __forceinline__ int range_shift(float most, float eps) {
  if (!(most < __builtin_inff())) return 0;
  const int e = (__builtin_amdgcn_frexp_expf(eps) + 1) >> 1;
  if (most == 0.f) return eps > 0.f ? -e : 0;
  const int m = __builtin_amdgcn_frexp_expf(most);
  return eps > 0.f && e > m ? -e : -m;
}
__device__ __forceinline__ float largest(const f32x4& v) {
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}

// y of 4 values from their n (or, gate_first, n'), the parameters and the gate
__device__ __forceinline__ f32x4 finish(const NormArgs& a, f32x4 n, const f32x4& w, const f32x4& b, const f32x4& z) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float v = fmaf(n[e], w[e], b[e]);
    if (a.gate && !a.gate_first)
      v *= a.silu ? silu(z[e]) : z[e];
    else if (!a.gate && a.silu)
      v = silu(v);
    n[e] = v;
  }
  return n;
}

// gi / groups and the remainder, by the host's ceil(2^32 / groups): the quotient is at most one too
// large for gi below 2^32.
__device__ __forceinline__ uint32_t row_of(uint32_t gi, const NormArgs& a, uint32_t& group) {
  if (a.groups == 1) {
    group = 0;
    return gi;
  }
  uint32_t row = __umulhi(gi, a.groups_inverse);
  int32_t rest = static_cast<int32_t>(gi - row * static_cast<uint32_t>(a.groups));
  const bool over = rest < 0;
  group = static_cast<uint32_t>(over ? rest + a.groups : rest);
  return over ? row - 1 : row;
}

template <typename TX, typename TY, int LPG, int V>
__global__ __launch_bounds__(kNormWaves* kWave) void norm_kernel(NormArgs a) {
  const uint32_t n_groups = static_cast<uint32_t>(a.rows) * static_cast<uint32_t>(a.groups);  // (at most 2^24)
  const uint32_t gi = (blockIdx.x * (kNormWaves * kWave) + threadIdx.x) / LPG;
  if (gi >= n_groups) return;  // whole groups of lanes; the others' sums stay among themselves
  const int c = threadIdx.x % LPG;
  uint32_t group;
  const uint32_t row = row_of(gi, a, group);
  const int64_t col = static_cast<int64_t>(group) * a.size;
  const TX* xp = static_cast<const TX*>(a.x) + row * a.x_stride + col;
  const int64_t zoff = row * a.gate_stride + col;
  const int64_t poff = a.shared ? 0 : col;
  f32x4 x[V], z[V], w[V], b[V];
#pragma unroll
  for (int t = 0; t < V; ++t) x[t] = load4u(xp, 4 * (c + LPG * t), a.size);
  if (a.gate) load_all<LPG>(a.gate, a.gate_bf16, zoff, c, a.size, z);
  if (a.weight) {
    load_all<LPG>(a.weight, a.param_bf16, poff, c, a.size, w);
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) w[t] = f32x4{1.f, 1.f, 1.f, 1.f};
  }
  if (a.bias) {
    load_all<LPG>(a.bias, a.param_bf16, poff, c, a.size, b);
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) b[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  const auto gate_x = [&]() {
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] *= a.silu ? silu(z[t][e]) : z[t][e];
  };
  const auto mean_square = [&]() {  // (x centred on the way)
    if (a.centered) {
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < V; ++t) sum += (x[t].x + x[t].y) + (x[t].z + x[t].w);
      const float mean = lanes_sum<LPG>(sum) * a.size_inverse;
#pragma unroll
      for (int t = 0; t < V; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] = 4 * (c + LPG * t) + e < a.size ? x[t][e] - mean : 0.f;
    }
    float sq = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sq = fmaf(x[t][e], x[t][e], sq);
    return lanes_sum<LPG>(sq) * a.size_inverse;
  };
  if (a.gate_first) gate_x();
  const float ms = mean_square() + a.eps;
  float rs = __builtin_amdgcn_rsqf(ms);
  if (!in_range(ms)) {  // (the group's lanes agree)
#pragma unroll
    for (int t = 0; t < V; ++t) x[t] = load4u(xp, 4 * (c + LPG * t), a.size);
    if (a.gate_first) gate_x();
    float most = 0.f;
#pragma unroll
    for (int t = 0; t < V; ++t) most = fmaxf(most, largest(x[t]));
#pragma unroll
    for (int m = 1; m < LPG; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
    const int sh = range_shift(most, a.eps);
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] = ldexpf(x[t][e], sh);
    rs = 1.0f / sqrtf(mean_square() + ldexpf(a.eps, 2 * sh));
  }
  TY* yp = static_cast<TY*>(a.y) + row * a.y_stride + col;
  // (one of three forms for the whole launch)
  if (a.gate && !a.gate_first) {
    if (a.silu) {
#pragma unroll
      for (int t = 0; t < V; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[t][e] = silu(z[t][e]);
    }
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] = fmaf(x[t][e] * rs, w[t][e], b[t][e]) * z[t][e];
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[t][e] = fmaf(x[t][e] * rs, w[t][e], b[t][e]);
    if (!a.gate && a.silu) {
#pragma unroll
      for (int t = 0; t < V; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[t][e] = silu(x[t][e]);
    }
  }
#pragma unroll
  for (int t = 0; t < V; ++t) store4u(yp, 4 * (c + LPG * t), a.size, x[t]);
}

// Groups beyond 2048 values: one workgroup a group, read once per sum and once for the result
// (from L2 after the first time).
template <typename TX, typename TY>
__global__ __launch_bounds__(kNormWaves* kWave) void norm_long_kernel(NormArgs a) {
  __shared__ float part[kNormWaves];
  const uint32_t gi = blockIdx.x;
  const int tid = threadIdx.x;
  uint32_t group;
  const uint32_t row = row_of(gi, a, group);
  const int64_t col = static_cast<int64_t>(group) * a.size;
  const TX* xp = static_cast<const TX*>(a.x) + row * a.x_stride + col;
  const int64_t zoff = row * a.gate_stride + col;
  const int64_t poff = a.shared ? 0 : col;
  int sh = 0;  // x counts 2^sh times
  const auto value = [&](int k, f32x4& z) {
    f32x4 x = load4u(xp, k, a.size);
    if (a.gate) z = load_any(a.gate, a.gate_bf16, zoff, k, a.size);
    if (a.gate_first)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= a.silu ? silu(z[e]) : z[e];
    if (sh != 0)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = ldexpf(x[e], sh);
    return x;
  };
  const auto gather = [&](float v) {  // a wave's value for the other waves
    __syncthreads();  // (the last one's readers are done)
    if (tid % kWave == 0) part[tid / kWave] = v;
    __syncthreads();
  };
  const auto total = [&](float v) {
    gather(lanes_sum<kWave>(v));
    return (part[0] + part[1]) + (part[2] + part[3]);
  };
  const float per = a.size_inverse;
  constexpr int step = 4 * kNormWaves * kWave;
  float mean = 0.f;
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  const auto mean_square = [&]() {
    if (a.centered) {
      float sum = 0.f;
      for (int k = 4 * tid; k < a.size; k += step) {
        const f32x4 x = value(k, z);
        sum += (x.x + x.y) + (x.z + x.w);
      }
      mean = total(sum) * per;
    }
    float sq = 0.f;
    for (int k = 4 * tid; k < a.size; k += step) {
      const f32x4 x = value(k, z);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = k + e < a.size ? x[e] - mean : 0.f;
        sq = fmaf(v, v, sq);
      }
    }
    return total(sq) * per;
  };
  const float ms = mean_square() + a.eps;
  float rs = __builtin_amdgcn_rsqf(ms);
  if (!in_range(ms)) {  // (the workgroup agrees)
    float most = 0.f;
    for (int k = 4 * tid; k < a.size; k += step) most = fmaxf(most, largest(value(k, z)));
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
    gather(most);
    sh = range_shift(largest(f32x4{part[0], part[1], part[2], part[3]}), a.eps);
    rs = 1.0f / sqrtf(mean_square() + ldexpf(a.eps, 2 * sh));
  }
  TY* yp = static_cast<TY*>(a.y) + row * a.y_stride + col;
  for (int k = 4 * tid; k < a.size; k += step) {
    f32x4 n = value(k, z);
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = (n[e] - mean) * rs;
    const f32x4 w = a.weight ? load_any(a.weight, a.param_bf16, poff, k, a.size) : f32x4{1.f, 1.f, 1.f, 1.f};
    const f32x4 b = a.bias ? load_any(a.bias, a.param_bf16, poff, k, a.size) : f32x4{0.f, 0.f, 0.f, 0.f};
    store4u(yp, k, a.size, finish(a, n, w, b, z));
  }
}

template <typename TX, typename TY, int LPG, int V>
hipError_t launch_v(const NormArgs& a, hipStream_t s) {
  const int64_t groups = static_cast<int64_t>(a.rows) * a.groups;
  constexpr int per = kNormWaves * kWave / LPG;
  norm_kernel<TX, TY, LPG, V><<<static_cast<unsigned>((groups + per - 1) / per), kNormWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t launch_t(const NormArgs& a, hipStream_t s) {
  // Two vectors a lane up to 512 values: 15717 x 32 groups of 128 take 95 us fp32 x and 88 us bf16 x, against
  // 94 / 94 us with one vector (twice the lanes, each with the group's fixed work) and 103 / 96 with four.
  if (a.size <= 32) return launch_v<TX, TY, 4, 2>(a, s);
  if (a.size <= 64) return launch_v<TX, TY, 8, 2>(a, s);
  if (a.size <= 128) return launch_v<TX, TY, 16, 2>(a, s);
  if (a.size <= 256) return launch_v<TX, TY, 32, 2>(a, s);
  if (a.size <= 512) return launch_v<TX, TY, 64, 2>(a, s);
  if (a.size <= 1024) return launch_v<TX, TY, 64, 4>(a, s);
  if (a.size <= 2048) return launch_v<TX, TY, 64, 8>(a, s);
  norm_long_kernel<TX, TY><<<static_cast<unsigned>(a.rows) * static_cast<unsigned>(a.groups), kNormWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

// A launch holds fewer than 2^32 threads: a call of more than 2^23 groups goes in pieces of rows
// (2^23 groups of 256 threads at most; a single row of 2^23 groups or more has groups of one or two
// values, 4 lanes each).
hipError_t launch_group_norm(const NormArgs& args, hipStream_t s) {
  const int32_t most = args.groups < (1 << 23) ? (1 << 23) / args.groups : 1;
  for (int32_t r = 0; r < args.rows;) {
    NormArgs a = args;
    a.groups_inverse = static_cast<uint32_t>(((1ull << 32) + args.groups - 1) / args.groups);  // (unused for one)
    a.size_inverse = 1.0f / static_cast<float>(args.size);
    a.rows = args.rows - r < most ? args.rows - r : most;
    const auto at = [r](const void* p, int bf16, int64_t stride) {
      return p ? static_cast<const char*>(p) + r * stride * (bf16 ? 2 : 4) : nullptr;
    };
    a.x = at(args.x, a.x_bf16, a.x_stride);
    a.gate = at(args.gate, a.gate_bf16, a.gate_stride);
    a.y = const_cast<char*>(at(args.y, a.y_bf16, a.y_stride));
    const hipError_t e = a.x_bf16 ? (a.y_bf16 ? launch_t<uint16_t, uint16_t>(a, s) : launch_t<uint16_t, float>(a, s))
                                  : (a.y_bf16 ? launch_t<float, uint16_t>(a, s) : launch_t<float, float>(a, s));
    if (e != hipSuccess) return e;
    r += a.rows;
  }
  return hipSuccess;
}

}  // namespace gdn
