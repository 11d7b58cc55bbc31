// Linear attention with a decay for each head, gfx950 (include/gdn.h, gdn_linear_prefill and
// gdn_linear_decode): S_t = e^g_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t over the slots' fp32 states.

#include "device_common.h"
#include "launch.h"

namespace gdn {
namespace {

typedef __attribute__((address_space(1))) f32x4 gf32x4;
typedef __attribute__((address_space(4))) const uint64_t cu64;
typedef __attribute__((address_space(4))) const float cfloat;

template <typename T>
__device__ __forceinline__ float value(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}

// (the hardware conversion: nearest even, and a NaN of any payload stays one)
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

__device__ __forceinline__ void put(void* o, int bf16, int64_t at, float v) {
  if (bf16) static_cast<uint16_t*>(o)[at] = to_bf16(v);
  else static_cast<float*>(o)[at] = v;
}

// ------------------------------------------------------------------------------ decode

constexpr int kDecodeWaves = 4;

// Workgroups go round-robin to the 8 XCDs: renumbered so that consecutive ones of a slot share an L2.
__device__ __forceinline__ int xcd_block() {
  const int n = gridDim.x, b = blockIdx.x;
  return n % 8 == 0 ? (b % 8) * (n / 8) + b / 8 : b;
}

// Bound by HBM: a state is read and written once, rows in any order, since
// o_r = scale (e^g S_r . q + v_r (k . q)) needs row r alone. A wave takes P passes of 1024 / D rows
// (4 KiB each); D / 16 lanes share a row, lane c holding the columns [4 c + D / 4 e, + 4), e < 4, and
// every load is issued before any arithmetic. Dots over a row's lanes are a fixed butterfly, so a
// slot's bits depend on nothing else in the call.
template <int D, int P, typename T>
__global__ __launch_bounds__(kDecodeWaves* kWave) void linear_decode_kernel(LinearArgs a) {
  constexpr int LPR = D / 16, RPP = kWave / LPR, PARTS = D / (RPP * P);
  const int lane = threadIdx.x & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int unit = xcd_block() * kDecodeWaves + w;
  if (unit >= a.hv * PARTS) return;
  const int j = unit / PARTS, i = blockIdx.y;
  const uint64_t sp = ((cu64*)a.state_ptrs)[i];
  if (sp == 0) return;
  const int h = j / a.group, c = lane % LPR, row0 = unit % PARTS * (RPP * P) + lane / LPR;
  gf32x4* S = (gf32x4*)(reinterpret_cast<float*>(sp) + static_cast<int64_t>(j) * D * D);
  f32x4 s[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[p][e] = __builtin_nontemporal_load(S + static_cast<int64_t>(row0 + p * RPP) * (D / 4) + c + LPR * e);
  const T* kp = static_cast<const T*>(a.k) + i * a.k_stride + h * D;
  const T* qp = static_cast<const T*>(a.q) + i * a.q_stride + h * D;
  typename Vec4<T>::Raw kr[4], qr[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kr[e] = Vec4<T>::load_raw(kp + 4 * (c + LPR * e));
    qr[e] = Vec4<T>::load_raw(qp + 4 * (c + LPR * e));
  }
  const T* vp = static_cast<const T*>(a.v) + i * a.v_stride + static_cast<int64_t>(j) * D;
  float vr[P];
#pragma unroll
  for (int p = 0; p < P; ++p) vr[p] = value(vp + row0 + p * RPP);
  const float decay = expf(((cfloat*)a.g)[i * a.g_stride + j]);
  float kq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int t = 0; t < 4; ++t) kq = fmaf(Vec4<T>::elem(kr[e], t), Vec4<T>::elem(qr[e], t), kq);
  kq = group_sum<LPR>(kq);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float sq = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f32x4 n;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        sq = fmaf(s[p][e][t], Vec4<T>::elem(qr[e], t), sq);
        n[t] = fmaf(vr[p], Vec4<T>::elem(kr[e], t), decay * s[p][e][t]);
      }
      __builtin_nontemporal_store(n, S + static_cast<int64_t>(row0 + p * RPP) * (D / 4) + c + LPR * e);
    }
    sq = group_sum<LPR>(sq);
    if (c == 0)
      put(a.o, a.o_bf16, (static_cast<int64_t>(i) * a.hv + j) * D + row0 + p * RPP, a.scale * fmaf(vr[p], kq, decay * sq));
  }
}

template <int D, int P, typename T>
hipError_t decode_units(const LinearArgs& a, int32_t m, hipStream_t s) {
  constexpr int PARTS = D / (kWave / (D / 16) * P);
  const dim3 grid(static_cast<unsigned>((a.hv * PARTS + kDecodeWaves - 1) / kDecodeWaves), static_cast<unsigned>(m));
  linear_decode_kernel<D, P, T><<<grid, kDecodeWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t decode_t(const LinearArgs& a, int32_t m, hipStream_t s) {
  const bool big = static_cast<int64_t>(m) * a.hv >= 1024;
  switch (a.d) {
    case 32: return decode_units<32, 1, T>(a, m, s);
    case 64: return big ? decode_units<64, 1, T>(a, m, s) : decode_units<64, 2, T>(a, m, s);
    default: return big ? decode_units<128, 1, T>(a, m, s) : decode_units<128, 2, T>(a, m, s);
  }
}

// ----------------------------------------------------------------------------- prefill

// The recurrence token by token: a workgroup a (sequence, v-head), 256 / D threads a state row.
template <int D, typename T>
__global__ __launch_bounds__(256) void linear_tokens_kernel(LinearArgs a, const int32_t* cu, int total) {
  constexpr int TPR = 256 / D, COLS = D / TPR;
  __shared__ float kq[2][D];
  const int j = blockIdx.x, i = blockIdx.y, h = j / a.group;
  const int row = threadIdx.x / TPR, c0 = threadIdx.x % TPR * COLS;
  const uint64_t sp = a.state_ptrs[i];
  if (sp == 0) return;
  const int lo = max(cu[i], 0), hi = min(cu[i + 1], total);
  if (lo >= hi) return;
  float* S = reinterpret_cast<float*>(sp) + (static_cast<int64_t>(j) * D + row) * D + c0;
  float s[COLS];
#pragma unroll
  for (int e = 0; e < COLS; ++e) s[e] = S[e];
  for (int64_t t = lo; t < hi; ++t) {
    __syncthreads();
    if (threadIdx.x < D) kq[0][threadIdx.x] = value(static_cast<const T*>(a.k) + t * a.k_stride + h * D + threadIdx.x);
    else if (threadIdx.x < 2 * D)
      kq[1][threadIdx.x - D] = value(static_cast<const T*>(a.q) + t * a.q_stride + h * D + threadIdx.x - D);
    const float v = value(static_cast<const T*>(a.v) + t * a.v_stride + static_cast<int64_t>(j) * D + row);
    const float f = expf(a.g[t * a.g_stride + j]);
    __syncthreads();
    float o = 0.f;
#pragma unroll
    for (int e = 0; e < COLS; ++e) {
      s[e] = fmaf(v, kq[0][c0 + e], f * s[e]);
      o = fmaf(s[e], kq[1][c0 + e], o);
    }
    o = group_sum<TPR>(o);
    if (threadIdx.x % TPR == 0) put(a.o, a.o_bf16, (t * a.hv + j) * D + row, a.scale * o);
  }
#pragma unroll
  for (int e = 0; e < COLS; ++e) S[e] = s[e];
}

template <typename T>
hipError_t prefill_t(const LinearArgs& a, const int32_t* cu, int32_t n, int32_t total, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.hv), static_cast<unsigned>(n));
  switch (a.d) {
    case 32: linear_tokens_kernel<32, T><<<grid, 256, 0, s>>>(a, cu, total); break;
    case 64: linear_tokens_kernel<64, T><<<grid, 256, 0, s>>>(a, cu, total); break;
    default: linear_tokens_kernel<128, T><<<grid, 256, 0, s>>>(a, cu, total); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_decode(const LinearArgs& a, int32_t m, hipStream_t s) {
  return a.bf16 ? decode_t<uint16_t>(a, m, s) : decode_t<float>(a, m, s);
}

size_t linear_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_linear_prefill(const LinearArgs& a, const int32_t* cu, int32_t n, int32_t total, void*, hipStream_t s) {
  return a.bf16 ? prefill_t<uint16_t>(a, cu, n, total, s) : prefill_t<float>(a, cu, n, total, s);
}

}  // namespace gdn
