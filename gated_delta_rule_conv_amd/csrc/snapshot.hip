// 8-bit snapshots of slots, gfx950: a state row x[d] becomes d codes of one byte and one fp32
// scale, scale = max|x| / M and code = round(x * (M * (1 / max|x|))), M = 127 (int8) or 448 (e4m3);
// read back x = scale * code. The conv state travels beside it as it is.
// ("qLLM", "What's still open", and aprender #5279, "Phase plan", P7: prefix reuse needs stored
// recurrent states; a fixed-size fp32 state is the largest thing such a store holds.)
//
// Bound by HBM: per state value 4 bytes one way and 1 byte the other, a few VALU operations. 64 slots
// of a 16/32-head, d = 128 layer pack in 31.4 us (175 MB, 5.6 TB/s) and unpack in 25.0 us (166 MB, 6.6 TB/s: the
// codes, 35 MB, come from the Infinity Cache where they were just written).
// A wave takes UN consecutive KiB of a state: in each, lane l holds values [4l, 4l + 4), so a
// row is d/4 adjacent lanes, loads and stores of fp32 are whole KiB, and the codes of a KiB are
// 256 contiguous bytes. The row maximum is an integer maximum of the magnitudes' bits over those
// lanes (bits of non-negative floats order as the floats do, infinity and NaN above all), so
// a NaN is never lost in it.

#include "device_common.h"
#include "launch.h"

namespace gdn {
namespace {

typedef __attribute__((address_space(1))) f32x4 gf32x4;
typedef __attribute__((address_space(1))) float gfloat;
typedef __attribute__((address_space(1))) uint32_t gu32;
typedef __attribute__((address_space(4))) const uint64_t cu64;
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kPackWaves = 4;  // waves per workgroup
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kTinyBits = (127u - 100u) << 23;  // 2^-100

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
  return v > o ? v : o;
}

// Maximum over aligned groups of L lanes (8, 16 or 32); every lane of the group gets it.
template <int L>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  v = dpp_umax<0xB1>(v);
  v = dpp_umax<0x4E>(v);
  v = dpp_umax<0x141>(v);
  if constexpr (L >= 16) v = dpp_umax<0x140>(v);
  if constexpr (L >= 32) {
    const uint32_t o = __shfl_xor(v, 16);
    v = v > o ? v : o;
  }
  return v;
}

// Copies the conv states, 4 KiB a workgroup.
__device__ __forceinline__ void copy_conv(const char* src, char* dst, int64_t bytes, int64_t block) {
  const int64_t k = block * (kPackWaves * kWave) + threadIdx.x;
  if (k * 16 < bytes) ((gf32x4*)reinterpret_cast<float*>(dst))[k] = ((const gf32x4*)reinterpret_cast<const float*>(src))[k];
}

template <int D, int UN, bool E4M3>
__global__ __launch_bounds__(kPackWaves* kWave) void pack_kernel(PackArgs a, int32_t state_blocks) {
  constexpr int L = D / 4;  // lanes per state row
  const int i = blockIdx.y;
  const uint64_t sp = ((cu64*)a.state_ptrs)[i];
  const uint64_t pp = ((cu64*)a.packed_ptrs)[i];
  const uint64_t cp = a.conv_ptrs ? ((cu64*)a.conv_ptrs)[i] : 0;
  if (sp == 0 || pp == 0 || (a.conv_ptrs && cp == 0)) return;
  char* block = reinterpret_cast<char*>(pp);
  const int64_t codes = static_cast<int64_t>(a.rows) * D;
  if (static_cast<int>(blockIdx.x) >= state_blocks) {
    copy_conv(reinterpret_cast<const char*>(cp), block + codes + static_cast<int64_t>(a.rows) * 4, a.conv_bytes,
              blockIdx.x - state_blocks);
    return;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t kib = (static_cast<int64_t>(blockIdx.x) * kPackWaves + w) * UN;  // first KiB of the wave
  const int64_t kibs = codes / 256;                                              // (whole: rows * d is a multiple of 1024)
  const gf32x4* src = (const gf32x4*)reinterpret_cast<const float*>(sp);
  f32x4 x[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (kib + u < kibs) x[u] = __builtin_nontemporal_load(src + (kib + u) * kWave + lane);
  constexpr float M = E4M3 ? 448.0f : 127.0f;
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    if (kib + u >= kibs) break;
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t b = __float_as_uint(x[u][e]) & 0x7FFFFFFFu;
      top = top > b ? top : b;
    }
    top = group_umax<L>(top);
    const bool live = top >= kTinyBits && top < kInfBits;
    const float amax = __uint_as_float(top);
    const float inv = M * (1.0f / (live ? amax : 1.0f));
    const float scale = live ? amax / M : top >= kInfBits ? __uint_as_float(0x7FC00000u) : 0.0f;
    uint32_t code = 0;
    if constexpr (E4M3) {
      int p = __builtin_amdgcn_cvt_pk_fp8_f32(x[u][0] * inv, x[u][1] * inv, 0, false);
      p = __builtin_amdgcn_cvt_pk_fp8_f32(x[u][2] * inv, x[u][3] * inv, p, true);
      code = static_cast<uint32_t>(p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = static_cast<int>(rintf(live ? x[u][e] * inv : 0.0f));
        code |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * e);
      }
    }
    if (!live) code = 0;
    const int64_t v = (kib + u) * kWave + lane;  // 4-value group of the state
    __builtin_nontemporal_store(code, (gu32*)reinterpret_cast<uint32_t*>(block) + v);
    if (lane % L == 0) ((gfloat*)reinterpret_cast<float*>(block + codes))[v / L] = scale;
  }
}

template <int D, int UN, bool E4M3>
__global__ __launch_bounds__(kPackWaves* kWave) void unpack_kernel(PackArgs a, int32_t state_blocks) {
  constexpr int L = D / 4;
  const int i = blockIdx.y;
  const uint64_t sp = ((cu64*)a.state_ptrs)[i];
  const uint64_t pp = ((cu64*)a.packed_ptrs)[i];
  const uint64_t cp = a.conv_ptrs ? ((cu64*)a.conv_ptrs)[i] : 0;
  if (sp == 0 || pp == 0 || (a.conv_ptrs && cp == 0)) return;
  const char* block = reinterpret_cast<const char*>(pp);
  const int64_t codes = static_cast<int64_t>(a.rows) * D;
  if (static_cast<int>(blockIdx.x) >= state_blocks) {
    copy_conv(block + codes + static_cast<int64_t>(a.rows) * 4, reinterpret_cast<char*>(cp), a.conv_bytes,
              blockIdx.x - state_blocks);
    return;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t kib = (static_cast<int64_t>(blockIdx.x) * kPackWaves + w) * UN;
  const int64_t kibs = codes / 256;
  const gu32* src = (const gu32*)reinterpret_cast<const uint32_t*>(block);
  const gfloat* scales = (const gfloat*)reinterpret_cast<const float*>(block + codes);
  gf32x4* dst = (gf32x4*)reinterpret_cast<float*>(sp);
  uint32_t code[UN];
  float scale[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (kib + u < kibs) {
      const int64_t v = (kib + u) * kWave + lane;
      code[u] = src[v];
      scale[u] = scales[v / L];
    }
#pragma unroll
  for (int u = 0; u < UN; ++u) {
    if (kib + u >= kibs) break;
    f32x4 x;
    if constexpr (E4M3) {
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(code[u], false);
      const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(code[u], true);
      x = f32x4{lo.x, lo.y, hi.x, hi.y};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = static_cast<float>(static_cast<int8_t>(code[u] >> (8 * e)));
    }
    x.x *= scale[u];
    x.y *= scale[u];
    x.z *= scale[u];
    x.w *= scale[u];
    __builtin_nontemporal_store(x, dst + (kib + u) * kWave + lane);
  }
}

template <int D, bool E4M3, bool UNPACK>
hipError_t launch_d(const PackArgs& a, int32_t n, hipStream_t s) {
  constexpr int UN = 4;
  const int64_t kibs = static_cast<int64_t>(a.rows) * D / 256;
  const int64_t per = static_cast<int64_t>(kPackWaves) * UN;
  const int32_t sb = static_cast<int32_t>((kibs + per - 1) / per);
  const int64_t per_conv = static_cast<int64_t>(kPackWaves) * kWave * 16;
  const int64_t cb = (a.conv_bytes + per_conv - 1) / per_conv;
  const dim3 grid(static_cast<unsigned>(sb + cb), static_cast<unsigned>(n));
  if constexpr (UNPACK)
    unpack_kernel<D, UN, E4M3><<<grid, kPackWaves * kWave, 0, s>>>(a, sb);
  else
    pack_kernel<D, UN, E4M3><<<grid, kPackWaves * kWave, 0, s>>>(a, sb);
  return hipGetLastError();
}

template <bool E4M3, bool UNPACK>
hipError_t launch_e(const PackArgs& a, int32_t n, hipStream_t s) {
  switch (a.d) {
    case 32: return launch_d<32, E4M3, UNPACK>(a, n, s);
    case 64: return launch_d<64, E4M3, UNPACK>(a, n, s);
    default: return launch_d<128, E4M3, UNPACK>(a, n, s);
  }
}

}  // namespace

hipError_t launch_slot_pack(const PackArgs& a, int32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  return a.e4m3 ? launch_e<true, false>(a, n, s) : launch_e<false, false>(a, n, s);
}

hipError_t launch_slot_unpack(const PackArgs& a, int32_t n, hipStream_t s) {
  if (n == 0) return hipSuccess;
  return a.e4m3 ? launch_e<true, true>(a, n, s) : launch_e<false, true>(a, n, s);
}

}  // namespace gdn
