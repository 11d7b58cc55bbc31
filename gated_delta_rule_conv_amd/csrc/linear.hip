// Linear attention with a decay for each head, gfx950 (include/gdn.h, gdn_linear_prefill and
// gdn_linear_decode): S_t = e^g_t S_{t-1} + v_t k_t^T, o_t = scale S_t q_t over the slots' fp32 states.

#include <type_traits>

#include "device_common.h"
#include "launch.h"
#include "mma.h"

#include "../../include/gdn.h"

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
// o_r = scale (e^g S_r . q + v_r (k . q)) needs row r alone. A wave takes 1024 / D rows (4 KiB); D / 16
// lanes share a row, lane c holding the columns [4 c + D / 4 e, + 4), e < 4, and every load is issued before any arithmetic.
// Dots over a row's lanes are a fixed butterfly, so a slot's bits depend on nothing else in the call. Twice the rows
// a wave: slower everywhere (32 heads, d = 128: 1 slot 4.8 us against 4.2, 64 slots 48.5 against 46.7, 256 slots 186 against
// 176, 6.1 TB/s).
template <int D, typename T>
__global__ __launch_bounds__(kDecodeWaves* kWave) void linear_decode_kernel(LinearArgs a) {
  constexpr int LPR = D / 16, ROWS = kWave / LPR, PARTS = D / ROWS;
  const int lane = threadIdx.x & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int unit = xcd_block() * kDecodeWaves + w;
  if (unit >= a.hv * PARTS) return;
  const int j = unit / PARTS, i = blockIdx.y;
  const uint64_t sp = ((cu64*)a.state_ptrs)[i];
  if (sp == 0) return;
  const int h = j / a.group, c = lane % LPR, row = unit % PARTS * ROWS + lane / LPR;
  gf32x4* S = (gf32x4*)(reinterpret_cast<float*>(sp) + (static_cast<int64_t>(j) * D + row) * D);
  f32x4 s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] = __builtin_nontemporal_load(S + c + LPR * e);
  const T* kp = static_cast<const T*>(a.k) + i * a.k_stride + h * D;
  const T* qp = static_cast<const T*>(a.q) + i * a.q_stride + h * D;
  typename Vec4<T>::Raw kr[4], qr[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kr[e] = Vec4<T>::load_raw(kp + 4 * (c + LPR * e));
    qr[e] = Vec4<T>::load_raw(qp + 4 * (c + LPR * e));
  }
  const float v = value(static_cast<const T*>(a.v) + i * a.v_stride + static_cast<int64_t>(j) * D + row);
  const float decay = expf(((cfloat*)a.g)[i * a.g_stride + j]);
  float kq = 0.f, sq = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f32x4 n;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float k = Vec4<T>::elem(kr[e], t), q = Vec4<T>::elem(qr[e], t);
      kq = fmaf(k, q, kq);
      sq = fmaf(s[e][t], q, sq);
      n[t] = fmaf(v, k, decay * s[e][t]);
    }
    __builtin_nontemporal_store(n, S + c + LPR * e);
  }
  kq = group_sum<LPR>(kq);
  sq = group_sum<LPR>(sq);
  if (c == 0) put(a.o, a.o_bf16, (static_cast<int64_t>(i) * a.hv + j) * D + row, a.scale * fmaf(v, kq, decay * sq));
}

template <int D, typename T>
hipError_t decode_dt(const LinearArgs& a, int32_t m, hipStream_t s) {
  constexpr int PARTS = D / (kWave / (D / 16));
  const dim3 grid(static_cast<unsigned>((a.hv * PARTS + kDecodeWaves - 1) / kDecodeWaves), static_cast<unsigned>(m));
  linear_decode_kernel<D, T><<<grid, kDecodeWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t decode_t(const LinearArgs& a, int32_t m, hipStream_t s) {
  switch (a.d) {
    case 32: return decode_dt<32, T>(a, m, s);
    case 64: return decode_dt<64, T>(a, m, s);
    default: return decode_dt<128, T>(a, m, s);
  }
}

// ----------------------------------------------------------------------------- prefill
//
// A sequence goes in chunks of 64 tokens from its own first one. With G_i the sum of g over a chunk's tokens up
// to i, n its last, and S the state before it:
//   o_i = scale (e^G_i S q_i + sum_{j <= i} e^(G_i - G_j) (q_i . k_j) v_j)
//   S  <- e^G_n S + sum_j e^(G_n - G_j) v_j k_j^T
// all four products on matrix cores. A workgroup takes a v-head of a tile, a run of a sequence's chunks; each of its
// waves owns 16 or 32 of the d_v columns of S^T [d_k][d_v] in accumulators, where they lie as a product's left operand wants
// them: lane l of a 16x16 tile's result holds rows 4 h + r (h = l / 16, r < 4) of column l % 16, so a step over 32 contracted values
// takes its values in the order 32 s + 16 u + 4 h + r (u < 2; fp32: 16 s + 4 h + r) from both operands, and S never passes through
// LDS. q is stored in LDS in that order, k, v as they came (read by rows for q . k, by columns, transposed on the way, for the
// state), the masked scores in that order again.
//
// Precision: with bf16 input every product has one operand that is exact in bf16. The other is fp32 and goes as three bf16
// thirds, x = a + b + c exactly (8 bits each, cut, not rounded): three products, no rounding but those of fp32 sums. (Two thirds
// alone, cut to 2^-15 of a term, would show where terms cancel, in bf16 outputs too.) fp32 input
// goes through fp32 products. Sums of g are kept in base 2 as a multiple of 2^-8, exact up to 2^16, and a rest, so that
// differences between tokens behind a strongly forgetting one keep their digits.
//
// Sequences are cut into tiles so that enough workgroups run: a first pass forms what each tile adds to the state, a scan the
// state before each tile, and the last pass runs all tiles at once. Tiles begin at a sequence's own first token.
//
// What bounds it (16 k-heads, 32 v-heads, d = 128, bf16): 4096 tokens, tiles of 4 chunks, 24 + 13 + 48 us; the pack of 15717
// tokens, fp32 outputs, tiles of 16, 54 + 15 + 164 us, where the bytes alone would take 111. No single thing bounds the last
// pass: per wave and chunk 240 matrix, 1300 to 1400 vector and 143 LDS instructions, which a SIMD's two waves issue mostly one at a
// time (a vector one every 5 cycles of a wave, LDS conflicts in 4 cycles of 10); leaving out stores, scores, loads or the
// state's update takes off 6 to 18% each. All 512 workgroups of the 4096 tokens run at once, two a CU (7.1 waves of 8 on
// average), a chunk of both in 20000 cycles. fp32 input: 4096 tokens 189 us, the pack 663, beside 56 and 214 for fp32 products of
// S q and v k^T alone; at d = 128 one workgroup a CU (320 registers, 117 KiB of LDS). Tried and slower: 8 waves of 16 columns (the pack 196 us against 180, 8-chunk tiles), vector
// instructions placed between matrix ones by scheduling groups (197 against 180).

constexpr int kChunk = 64;
constexpr float kForget = -128.0f;  // e^-128 is 0 in fp32
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ void barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The same number, to be taken as another one each time: what is computed from it is not kept in registers over a
// loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Sum over the wave's lanes up to each one.
__device__ __forceinline__ float wave_scan(float v) {
  const auto add = [&](auto moved) { v += __int_as_float(moved); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xF, 0xF, false));  // row_shr 1, 2, 4, 8
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));  // lane 15 of a row to the next row
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));  // lane 31 to the upper rows
  return v;
}

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// Products of an input's values (bf16 or fp32), exact, with fp32 numbers.
template <typename T>
struct Prod;

template <>
struct Prod<uint16_t> {
  static constexpr int STEP = 32, PER = 8;  // contracted values a step, a lane's of them
  typedef bf16x8 Exact;
  struct Full {
    bf16x8 a, b, c;
  };
  // the high halves of two words
  __device__ __forceinline__ static uint32_t tops(uint32_t lo, uint32_t hi) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }
  __device__ __forceinline__ static void thirds(float x, uint32_t& a, uint32_t& b, uint32_t& c) {
    a = __float_as_uint(x);
    const float r = x - __uint_as_float(a & 0xFFFF0000u);
    b = __float_as_uint(r);
    c = __float_as_uint(r - __uint_as_float(b & 0xFFFF0000u));
  }
  __device__ __forceinline__ static Full full(const float (&x)[8]) {
    u32x4 a, b, c;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t a0, b0, c0, a1, b1, c1;
      thirds(x[2 * e], a0, b0, c0);
      thirds(x[2 * e + 1], a1, b1, c1);
      a[e] = tops(a0, a1);
      b[e] = tops(b0, b1);
      c[e] = tops(c0, c1);
    }
    return Full{__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, c)};
  }
  __device__ __forceinline__ static float value(const Exact& x, int e) { return static_cast<float>(x[e]); }
  __device__ __forceinline__ static void clear(Exact& x, int e) { x[e] = static_cast<__bf16>(0.f); }
  // whether one of them is an infinity or a NaN
  __device__ __forceinline__ static bool odd(const Exact& x) {
    const u32x4 y = __builtin_bit_cast(u32x4, x);
    uint32_t o = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) o |= (y[e] & 0x7F807F80u) + 0x00800080u;
    return (o & 0x80008000u) != 0;
  }
  __device__ __forceinline__ static Full load(const uint16_t* p, int plane) {
    return Full{*reinterpret_cast<const bf16x8*>(p), *reinterpret_cast<const bf16x8*>(p + plane),
                *reinterpret_cast<const bf16x8*>(p + 2 * plane)};
  }
  __device__ __forceinline__ static f32x4 exact(const Exact& a, const Exact& b, const f32x4& acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
  }
  // one of the three products of a full operand, the smallest first
  static constexpr int PARTS = 3;
  __device__ __forceinline__ static const bf16x8& part(const Full& f, int p) { return p == 0 ? f.c : p == 1 ? f.b : f.a; }
  __device__ __forceinline__ static f32x4 left(const Full& a, const Exact& b, const f32x4& acc, int p) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(part(a, p), b, acc, 0, 0, 0);
  }
  __device__ __forceinline__ static f32x4 right(const Exact& a, const Full& b, const f32x4& acc, int p) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, part(b, p), acc, 0, 0, 0);
  }
};

template <>
struct Prod<float> {
  static constexpr int STEP = 16, PER = 4;
  typedef f32x4 Exact;
  typedef f32x4 Full;
  __device__ __forceinline__ static Full full(const float (&x)[4]) { return f32x4{x[0], x[1], x[2], x[3]}; }
  __device__ __forceinline__ static float value(const Exact& x, int e) { return x[e]; }
  __device__ __forceinline__ static void clear(Exact& x, int e) { x[e] = 0.f; }
  __device__ __forceinline__ static bool odd(const Exact& x) {
    return !(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))) < __builtin_inff()) || x[0] != x[0] ||
           x[1] != x[1] || x[2] != x[2] || x[3] != x[3];
  }
  __device__ __forceinline__ static Full load(const float* p, int) { return *reinterpret_cast<const f32x4*>(p); }
  __device__ __forceinline__ static f32x4 exact(const Exact& a, const Exact& b, f32x4 acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
    return acc;
  }
  static constexpr int PARTS = 4;
  __device__ __forceinline__ static f32x4 left(const Full& a, const Exact& b, const f32x4& acc, int p) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a[p], b[p], acc, 0, 0, 0);
  }
  __device__ __forceinline__ static f32x4 right(const Exact& a, const Full& b, const f32x4& acc, int p) {
    return left(a, b, acc, p);
  }
};

// Where a tile lies.
struct Place {
  int seq;   // -1: there is no such tile
  int part;  // which of its sequence's
  int slot;  // its room for a state in the workspace; -1: the only tile of its sequence
};

struct LinearPlan {
  const int32_t* cu;
  int32_t n;
  int32_t total;
  int32_t tokens;      // a tile's
  const Place* tiles;  // by tile and (slots) by room; null: found by the workgroup
  const Place* slots;
  float* states;       // [rooms][hv][D][D]
  float* kept;         // [rooms][hv]: e^(sum of g)
  int32_t first;       // the launch's first tile
};

__device__ __forceinline__ void sequence(const LinearPlan& p, int i, int& lo, int& hi) {
  lo = max(p.cu[i], 0);
  hi = max(min(p.cu[i + 1], p.total), lo);
}

// How many tiles a sequence has: up to 5 chunks are one, whatever a tile's length (a tile of 2 chunks each for 256 tokens of
// one sequence: 31.5 us against 26.2 in one, 32 heads, d = 128; for 384: 33.8 against 35.5).
constexpr int kUncut = 5 * kChunk;
__device__ __forceinline__ int tiles_of(const LinearPlan& p, int len) {
  return len <= kUncut ? len > 0 : len / p.tokens + (len % p.tokens != 0);
}

// Tile b, or with SLOTS the tile of room b, by a scan over the sequences, 64 at a time.
template <bool SLOTS>
__device__ Place find_place(const LinearPlan& p, int b) {
  const int lane = threadIdx.x & (kWave - 1);
  int tiles = 0, rooms = 0;
  for (int i0 = 0; i0 < p.n; i0 += kWave) {
    int lo = 0, hi = 0;
    if (i0 + lane < p.n) sequence(p, i0 + lane, lo, hi);
    const int t = tiles_of(p, hi - lo), r = t > 1 ? t : 0;
    int ts = t, rs = r;
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
      const int a = __shfl_up(ts, m), c = __shfl_up(rs, m);
      if (lane >= m) {
        ts += a;
        rs += c;
      }
    }
    const int from = SLOTS ? rooms + rs - r : tiles + ts - t, here = SLOTS ? r : t;
    const uint64_t hit = __ballot(b >= from && b < from + here);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int part = b - __shfl(from, l), room = rooms + __shfl(rs - r, l);
      return Place{i0 + l, part, __shfl(r, l) ? room + part : -1};
    }
    tiles += __shfl(ts, kWave - 1);
    rooms += __shfl(rs, kWave - 1);
  }
  return Place{-1, 0, -1};
}

template <bool SLOTS>
__device__ __forceinline__ Place place_of(const LinearPlan& p, int b) {
  const Place* table = SLOTS ? p.slots : p.tiles;
  Place w = table ? table[b] : find_place<SLOTS>(p, b);
  w.seq = __builtin_amdgcn_readfirstlane(w.seq);
  w.part = __builtin_amdgcn_readfirstlane(w.part);
  w.slot = __builtin_amdgcn_readfirstlane(w.slot);
  return w;
}

// Both tables, for calls of many sequences: one workgroup, 1024 sequences at a time.
constexpr int kTableThreads = 1024;
__global__ __launch_bounds__(kTableThreads) void linear_table_kernel(LinearPlan p, Place* tiles, int n_tiles, Place* slots,
                                                                     int n_slots) {
  __shared__ int part[2][kTableThreads / kWave];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
  int t0 = 0, r0 = 0;
  for (int i0 = 0; i0 < p.n; i0 += kTableThreads) {
    const int i = i0 + tid;
    int lo = 0, hi = 0;
    if (i < p.n) sequence(p, i, lo, hi);
    const int t = tiles_of(p, hi - lo), r = t > 1 ? t : 0;
    int ts = t, rs = r;
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) {
      const int a = __shfl_up(ts, m), c = __shfl_up(rs, m);
      if (lane >= m) {
        ts += a;
        rs += c;
      }
    }
    __syncthreads();
    if (lane == kWave - 1) {
      part[0][w] = ts;
      part[1][w] = rs;
    }
    __syncthreads();
    int at = t0 + ts - t, room = r0 + rs - r;
    for (int v = 0; v < kTableThreads / kWave; ++v) {
      if (v < w) {
        at += part[0][v];
        room += part[1][v];
      }
      t0 += part[0][v];
      r0 += part[1][v];
    }
    for (int k = 0; k < t; ++k) {
      if (at + k < n_tiles) tiles[at + k] = Place{i, k, r ? room + k : -1};
      if (r && room + k < n_slots) slots[room + k] = Place{i, k, room + k};
    }
  }
  for (int b = t0 + tid; b < n_tiles; b += kTableThreads) tiles[b] = Place{-1, 0, -1};
  for (int b = r0 + tid; b < n_slots; b += kTableThreads) slots[b] = Place{-1, 0, -1};
}

// OUT: the pass with outputs.
template <int D, typename T, bool OUT>
struct LinearCfg {
  static constexpr int WAVES = D == 32 ? 2 : OUT ? 4 : D / 16, THREADS = WAVES * kWave;
  static constexpr int COLS = D / WAVES;    // d_v a wave
  static constexpr int VT = COLS / 16;      // 16x16 tiles: of d_v a wave
  static constexpr int KT = D / 16;         // of d_k
  static constexpr int STEP = Prod<T>::STEP;
  static constexpr int DS = D / STEP;       // steps over d
  static constexpr int JS = kChunk / STEP;  // and over tokens
  static constexpr int EPP = 16 / sizeof(T);        // values in 16 bytes
  static constexpr int PPR = D / EPP;               // 16-byte pieces a row
  static constexpr int PIECES = kChunk * PPR / THREADS;
  // Rows of tiles are 16 bytes longer than their values, which spreads 16 rows' pieces of 16 bytes over all banks.
  static constexpr int PITCH = D + EPP;
  static constexpr int PROWS = kChunk + EPP;  // of the scores
};

// OUT: outputs and the state behind the tile; else what the tile adds to the state.
template <int D, typename T, typename O, bool OUT>
__global__ __launch_bounds__((LinearCfg<D, T, OUT>::THREADS), (sizeof(T) == 2 ? OUT ? 2 : 4 : 1)) void linear_chunks_kernel(LinearArgs a,
                                                                                                                LinearPlan p) {
  using C = LinearCfg<D, T, OUT>;
  using P = Prod<T>;
  using Exact = typename P::Exact;
  using Full = typename P::Full;
  constexpr int PITCH = C::PITCH, PROWS = C::PROWS;
  constexpr int PLANES = sizeof(T) == 2 ? 3 : 1;  // of the scores
  __shared__ __attribute__((aligned(16))) T kl[kChunk * PITCH];
  __shared__ __attribute__((aligned(16))) T vl[kChunk * PITCH];
  __shared__ __attribute__((aligned(16))) T ql[OUT ? kChunk * PITCH : 16];
  __shared__ __attribute__((aligned(16))) T pl[OUT ? PLANES * kChunk * PROWS : 16];
  __shared__ __attribute__((aligned(16))) float gl[4][kChunk];  // G's multiple of 2^-8, its rest, scale e^G_i, e^(G_n - G_i)
  const int tid = threadIdx.x, lane = tid & (kWave - 1), w = __builtin_amdgcn_readfirstlane(tid / kWave);
  int l16 = lane & 15, h = lane >> 4, h4 = 4 * h;
  const int b = blockIdx.x % a.hv, tile = p.first + blockIdx.x / a.hv;
  // workgroups go round-robin to the 8 XCDs: neighbouring heads, which share k and q, to one of them
  const int j = a.hv % 8 == 0 ? (b % 8) * (a.hv / 8) + b / 8 : b;
  const Place at = place_of<!OUT>(p, tile);
  if (at.seq < 0) return;
  const uint64_t sp = a.state_ptrs[at.seq];
  if (sp == 0) return;
  int lo, hi;
  sequence(p, at.seq, lo, hi);
  lo = __builtin_amdgcn_readfirstlane(lo);
  hi = __builtin_amdgcn_readfirstlane(hi);
  const bool last = at.slot < 0 || hi - lo <= (at.part + 1) * static_cast<int64_t>(p.tokens);
  if (!OUT && last) return;  // (no tile follows)
  const int start = at.slot < 0 ? lo : lo + at.part * p.tokens, end = last ? hi : start + p.tokens;
  const int kh = j / a.group;
  const int64_t head = static_cast<int64_t>(j) * D * D;
  float* own = reinterpret_cast<float*>(sp) + head;
  float* room = at.slot < 0 ? nullptr : p.states + static_cast<int64_t>(at.slot) * a.hv * D * D + head;
  const int c0 = w * C::COLS;

  f32x4 s[C::KT][C::VT];
  if constexpr (OUT) {
    const float* from = room ? room : own;
#pragma unroll
    for (int t = 0; t < C::VT; ++t)
#pragma unroll
      for (int k = 0; k < C::KT; ++k)
        s[k][t] = *reinterpret_cast<const f32x4*>(from + (c0 + 16 * t + l16) * D + 16 * k + h4);
    // score tiles above the diagonal inside a step stay zero
    if constexpr (sizeof(T) == 2) {
      for (int x = tid; x < PLANES * 2 * 16 * 8; x += C::THREADS) {
        const int plane = x / 256, r = x % 256 / 8, h = x % 8 / 2, half = x % 2;  // 4 bytes each
        const int i = r < 16 ? r : 32 + r - 16, pos = (r < 16 ? 0 : 32) + 8 * h + 4 + 2 * half;
        *reinterpret_cast<uint32_t*>(pl + (plane * kChunk + i) * PROWS + pos) = 0;
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < C::VT; ++t)
#pragma unroll
      for (int k = 0; k < C::KT; ++k) s[k][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // --- a chunk's rows into registers, then into LDS
  u32x4 kr[C::PIECES], vr[C::PIECES], qr[OUT ? C::PIECES : 1];
  float gr = 0.f;
  int row0 = tid / C::PPR, piece = tid % C::PPR;
  constexpr int ROWS_UP = C::THREADS / C::PPR;
  typedef __attribute__((address_space(1))) const char gchar;
  typedef __attribute__((address_space(1))) const u32x4 gu32x4;
  typedef __attribute__((address_space(1))) const float gfloat;
  // (rows of a chunk at 32-bit offsets from its first: strides are below 2^24 bytes)
  gchar* kb = (gchar*)(static_cast<const T*>(a.k) + kh * D);
  gchar* qb = (gchar*)(static_cast<const T*>(a.q) + kh * D);
  gchar* vb = (gchar*)(static_cast<const T*>(a.v) + static_cast<int64_t>(j) * D);
  const int ks = static_cast<int>(a.k_stride * sizeof(T)), qs = static_cast<int>(a.q_stride * sizeof(T)),
            vs = static_cast<int>(a.v_stride * sizeof(T)), gs = static_cast<int>(a.g_stride * 4);
  gchar *kt = kb, *vt = vb, *qt = qb;
  int rows_there = 0;
  const auto aim = [&](int t, int len) {  // the next loads are of the chunk at t
    kt = kb + static_cast<int64_t>(t) * ks;
    vt = vb + static_cast<int64_t>(t) * vs;
    qt = qb + static_cast<int64_t>(t) * qs;
    rows_there = len - 1;
    gr = *(gfloat*)((gchar*)(a.g + t * a.g_stride + j) + __umul24(min(lane, len - 1), gs));
  };
  const auto load = [&](int u) {
    const uint32_t r = min(row0 + u * ROWS_UP, rows_there);
    kr[u] = *(gu32x4*)(kt + (__umul24(r, ks) + piece * 16));
    vr[u] = *(gu32x4*)(vt + (__umul24(r, vs) + piece * 16));
    if constexpr (OUT) qr[u] = *(gu32x4*)(qt + (__umul24(r, qs) + piece * 16));
  };
  float total_hi = 0.f, total_lo = 0.f;
  const auto put_rows = [&](auto whole, int len) {
#pragma unroll
    for (int u = 0; u < C::PIECES; ++u) {
      const int r = row0 + u * ROWS_UP;
      const bool there = decltype(whole)::value || r < len;
      const u32x4 zero = {0, 0, 0, 0};
      *reinterpret_cast<u32x4*>(kl + r * PITCH + piece * C::EPP) = there ? kr[u] : zero;
      *reinterpret_cast<u32x4*>(vl + r * PITCH + piece * C::EPP) = there ? vr[u] : zero;
      if constexpr (OUT) {
        const u32x4 q = there ? qr[u] : zero;
        if constexpr (sizeof(T) == 2) {  // values 8 p .. + 7 of 32: h = 2 (p % 2) and the next, u = p / 2
          T* to = ql + r * PITCH + 32 * (piece / 4) + 16 * (piece % 2) + 4 * (piece % 4 / 2);
          *reinterpret_cast<u32x2*>(to) = u32x2{q[0], q[1]};
          *reinterpret_cast<u32x2*>(to + 8) = u32x2{q[2], q[3]};
        } else {
          *reinterpret_cast<u32x4*>(ql + r * PITCH + piece * C::EPP) = q;
        }
      }
    }
  };
  const auto stage = [&](int len) {
    if (len == kChunk) put_rows(std::true_type{}, len);
    else put_rows(std::false_type{}, len);
    if (w == 0) {
      const float x = lane < len ? (gr < kForget ? kForget : gr) * kLog2e : 0.f;  // (a NaN stays)
      const float whole = rintf(x * 256.f) * 0x1p-8f;
      const float gh = wave_scan(whole), gt = wave_scan(x - whole);
      const float nh = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gh), kWave - 1));
      const float nt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gt), kWave - 1));
      gl[0][lane] = gh;
      gl[1][lane] = gt;
      gl[2][lane] = exp2_hw(gh + gt) * a.scale;
      gl[3][lane] = exp2_hw((nh - gh) + (nt - gt));
    }
  };
  // --- operands from LDS
  const auto k_row = [&](int i, int st) {  // row i of k, step st over d
    if constexpr (sizeof(T) == 2) {
      const T* f = kl + i * PITCH + 32 * st + h4;
      const u32x2 x = *reinterpret_cast<const u32x2*>(f), y = *reinterpret_cast<const u32x2*>(f + 16);
      return __builtin_bit_cast(Exact, u32x4{x[0], x[1], y[0], y[1]});
    } else {
      return *reinterpret_cast<const Exact*>(kl + i * PITCH + 16 * st + h4);
    }
  };
  const auto q_row = [&](int i, int st) {
    return *reinterpret_cast<const Exact*>(ql + i * PITCH + (sizeof(T) == 2 ? 32 * st + 2 * h4 : 16 * st + h4));
  };
  const auto column = [&](const T* tl, int c, int st) {  // columns c + l16 of k or v, step st over tokens
    if constexpr (sizeof(T) == 2) {
      const T* f = tl + (32 * st + h4 + (l16 >> 2)) * PITCH + c + 4 * (l16 & 3);
      const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(f));
      const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(f + 16 * PITCH));
      const i16x8 z = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
      return __builtin_bit_cast(Exact, z);
    } else {
      Exact z;
#pragma unroll
      for (int r = 0; r < 4; ++r) z[r] = tl[(16 * st + h4 + r) * PITCH + c + l16];
      return z;
    }
  };

  f32x4 o[OUT ? 4 : 1][C::VT];  // o^T: rows d_v, columns tokens 16 i + l16
  const auto store = [&](int at, int len) {
    if constexpr (OUT) {
      typedef __attribute__((address_space(1))) char gout;
      typedef __attribute__((address_space(1))) f32x4 go4;
      typedef __attribute__((address_space(1))) u32x2 go2;
      gout* ob = (gout*)a.o + ((static_cast<int64_t>(at) * a.hv + j) * D + c0) * sizeof(O);
      const int mine = l16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (16 * i + mine >= len) continue;
        const uint32_t to = __umul24(16 * i + mine, a.hv * D) + h4;
#pragma unroll
        for (int t = 0; t < C::VT; ++t) {
          const f32x4 v = o[i][t];
          if constexpr (sizeof(O) == 2) {
            const u32x2 x = {static_cast<uint32_t>(to_bf16(v[0])) | static_cast<uint32_t>(to_bf16(v[1])) << 16,
                             static_cast<uint32_t>(to_bf16(v[2])) | static_cast<uint32_t>(to_bf16(v[3])) << 16};
            *(go2*)(ob + (to + 16 * t) * 2) = x;
          } else {
            *(go4*)(ob + (to + 16 * t) * 4) = v;
          }
        }
      }
    }
  };

  const auto span = [&](int t) { return min(kChunk, end - t); };
  aim(start, span(start));
#pragma unroll
  for (int u = 0; u < C::PIECES; ++u) load(u);
  barrier_lds();
  for (int t = start; t < end;) {
    const int len = span(t);
    // (addresses are formed anew in every chunk: kept over the loop they would cost the registers of two waves a SIMD)
    l16 = fresh(l16);
    h = fresh(h);
    h4 = 4 * h;
    row0 = fresh(row0);
    piece = fresh(piece);
    stage(len);
    barrier_lds();
    const bool more = t + len < end;
    aim(more ? t + len : t, more ? span(t + len) : len);  // (loads without a branch: past the end, the same rows again)
    const float kept = exp2_hw(gl[0][kChunk - 1] + gl[1][kChunk - 1]);
    if constexpr (OUT) {
      // scores of tokens j (rows) for tokens i (columns), 10 tiles on and below the diagonal, side by side
      constexpr int SIDE = (10 + C::WAVES - 1) / C::WAVES;
      f32x4 acc[SIDE];
      int ti[SIDE], tj[SIDE];
#pragma unroll
      for (int y = 0; y < SIDE; ++y) {
        const int x = min(w + y * C::WAVES, 9);
        ti[y] = x >= 6 ? 3 : x >= 3 ? 2 : x >= 1 ? 1 : 0;
        tj[y] = x - ti[y] * (ti[y] + 1) / 2;
        acc[y] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int st = 0; st < C::DS; ++st)
#pragma unroll
        for (int y = 0; y < SIDE; ++y) acc[y] = P::exact(k_row(16 * tj[y] + l16, st), q_row(16 * ti[y] + l16, st), acc[y]);
#pragma unroll
      for (int y = 0; y < SIDE; ++y) {
        const int i = 16 * ti[y] + l16, j0 = 16 * tj[y] + h4;
        const float gi = gl[0][i], ri = gl[1][i];
        const f32x4 gj = *reinterpret_cast<const f32x4*>(&gl[0][j0]), rj = *reinterpret_cast<const f32x4*>(&gl[1][j0]);
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = acc[y][r] * (exp2_hw((gi - gj[r]) + (ri - rj[r])) * a.scale);
          asm volatile("" : "+v"(x));  // (formed in every lane: a branch around it costs more)
          v[r] = j0 + r <= i ? x : 0.f;
        }
        if (w + y * C::WAVES > 9) continue;
        if constexpr (sizeof(T) == 2) {
          uint32_t x3[3][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) P::thirds(v[r], x3[0][r], x3[1][r], x3[2][r]);
          T* to = pl + i * PROWS + 32 * (tj[y] / 2) + 2 * h4 + 4 * (tj[y] % 2);
#pragma unroll
          for (int z = 0; z < PLANES; ++z)
            *reinterpret_cast<u32x2*>(to + z * kChunk * PROWS) = u32x2{P::tops(x3[z][0], x3[z][1]), P::tops(x3[z][2], x3[z][3])};
        } else {
          *reinterpret_cast<f32x4*>(pl + i * PROWS + j0) = f32x4{v[0], v[1], v[2], v[3]};
        }
      }
      // e^G_i S q_i, the next chunk's loads between its steps
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < C::VT; ++t) o[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
      Exact q[2][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[0][i] = q_row(16 * i + l16, 0);
#pragma unroll
      for (int st = 0; st < C::DS; ++st) {
        if (st + 1 < C::DS)
#pragma unroll
          for (int i = 0; i < 4; ++i) q[(st + 1) % 2][i] = q_row(16 * i + l16, st + 1);
#pragma unroll
        for (int u = st; u < C::PIECES; u += C::DS) load(u);
        Full sf[C::VT];
#pragma unroll
        for (int t = 0; t < C::VT; ++t) {
          float x[P::PER];
#pragma unroll
          for (int e = 0; e < P::PER; ++e) x[e] = s[st * (C::STEP / 16) + e / 4][t][e % 4];
          sf[t] = P::full(x);
        }
#pragma unroll
        for (int part = 0; part < P::PARTS; ++part)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < C::VT; ++t) o[i][t] = P::left(sf[t], q[st % 2][i], o[i][t], part);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = gl[2][16 * i + l16];
#pragma unroll
        for (int t = 0; t < C::VT; ++t) o[i][t] = o[i][t] * f;
      }
      barrier_lds();
      // the scores times v
      int first[C::VT];  // the first token whose v is an infinity or a NaN in the lane's column
#pragma unroll
      for (int t = 0; t < C::VT; ++t) first[t] = kChunk;
      bool any = false;
#pragma unroll
      for (int st = 0; st < C::JS; ++st) {
        Exact v[C::VT];
        bool odd = false;
#pragma unroll
        for (int t = 0; t < C::VT; ++t) {
          v[t] = column(vl, c0 + 16 * t, st);
          odd |= P::odd(v[t]);
        }
        if (__ballot(odd)) {  // left out of the products: a score of 0 would not keep it from the tokens before it
          any = true;
#pragma unroll
          for (int t = 0; t < C::VT; ++t)
#pragma unroll
            for (int e = 0; e < P::PER; ++e)
              if (!(fabsf(P::value(v[t], e)) < __builtin_inff())) {
                first[t] = min(first[t], C::STEP * st + 16 * (e / 4) + h4 + e % 4);
                P::clear(v[t], e);
              }
        }
#pragma unroll
        for (int i = st * (C::STEP / 16); i < 4; ++i) {
          const Full sc = P::load(pl + (16 * i + l16) * PROWS + (sizeof(T) == 2 ? 32 * st + 2 * h4 : 16 * st + h4), kChunk * PROWS);
#pragma unroll
          for (int part = 0; part < P::PARTS; ++part)
#pragma unroll
            for (int t = 0; t < C::VT; ++t) o[i][t] = P::right(v[t], sc, o[i][t], part);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (any) {
#pragma unroll
        for (int t = 0; t < C::VT; ++t) {
          int f = min(first[t], __shfl_xor(first[t], 16));
          f = min(f, __shfl_xor(f, 32));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int from = __shfl(f, h4 + r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * i + l16 >= from) o[i][t][r] = __builtin_nanf("");
          }
        }
      }
      store(t, len);
    } else {
#pragma unroll
      for (int u = 0; u < C::PIECES; ++u) load(u);
    }
    // the state
#pragma unroll
    for (int k = 0; k < C::KT; ++k)
#pragma unroll
      for (int t = 0; t < C::VT; ++t) s[k][t] = s[k][t] * kept;
#pragma unroll
    for (int st = 0; st < C::JS; ++st) {
      float f[P::PER];
#pragma unroll
      for (int u = 0; u < P::PER / 4; ++u) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(&gl[3][C::STEP * st + 16 * u + h4]);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[4 * u + r] = x[r];
      }
      Full vf[C::VT];
#pragma unroll
      for (int t = 0; t < C::VT; ++t) {
        const Exact v = column(vl, c0 + 16 * t, st);
        float x[P::PER];
#pragma unroll
        for (int e = 0; e < P::PER; ++e) x[e] = P::value(v, e) * f[e];
        vf[t] = P::full(x);
      }
      Exact kc[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) kc[0][k] = column(kl, 16 * k, st);
#pragma unroll
      for (int k = 0; k < C::KT; k += 2) {
        if (k + 2 < C::KT)
#pragma unroll
          for (int x = 0; x < 2; ++x) kc[(k / 2 + 1) % 2][x] = column(kl, 16 * (k + 2 + x), st);
#pragma unroll
        for (int part = 0; part < P::PARTS; ++part)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int t = 0; t < C::VT; ++t) s[k + x][t] = P::right(kc[k / 2 % 2][x], vf[t], s[k + x][t], part);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    total_hi += gl[0][kChunk - 1];
    total_lo += gl[1][kChunk - 1];
    barrier_lds();
    t += len;
  }
  float* to = OUT ? own : room;
  if (OUT && !last) return;
#pragma unroll
  for (int t = 0; t < C::VT; ++t)
#pragma unroll
    for (int k = 0; k < C::KT; ++k) *reinterpret_cast<f32x4*>(to + (c0 + 16 * t + l16) * D + 16 * k + h4) = s[k][t];
  if (!OUT && tid == 0) p.kept[static_cast<int64_t>(at.slot) * a.hv + j] = exp2_hw(total_hi + total_lo);
}

// The state before each tile of the sequences that have several, from what the tiles add: in place.
constexpr int kScanThreads = 256;
template <int D>
__global__ __launch_bounds__(kScanThreads) void linear_scan_kernel(LinearArgs a, LinearPlan p) {
  constexpr int BLOCKS = D * D / 4 / kScanThreads;  // workgroups a head, 4 values a thread
  const int b = blockIdx.x % (a.hv * BLOCKS), j = b / BLOCKS;
  const Place at = place_of<true>(p, p.first + blockIdx.x / (a.hv * BLOCKS));
  if (at.seq < 0 || at.part != 0) return;
  const uint64_t sp = a.state_ptrs[at.seq];
  if (sp == 0) return;
  int lo, hi;
  sequence(p, at.seq, lo, hi);
  const int n = tiles_of(p, hi - lo);
  const int64_t e = static_cast<int64_t>(j) * (D * D / 4) + b % BLOCKS * kScanThreads + threadIdx.x;
  const int64_t up = static_cast<int64_t>(a.hv) * (D * D / 4);
  f32x4 z = reinterpret_cast<const f32x4*>(sp)[e];
  f32x4* to = reinterpret_cast<f32x4*>(p.states) + at.slot * up + e;
  const float* kept = p.kept + static_cast<int64_t>(at.slot) * a.hv + j;
  // Two tiles at a time, the next two on their way (the last tile added nothing). One at a time: 8 heads, d = 64, 64 tiles of
  // 256 tokens 25.6 us against 16.0, 32 heads, d = 128, 16 of 1024 23.1 against 24.0; four at a time: the latter 26.5.
  constexpr int A = 2;
  f32x4 added[A], next[A];
  float f[A], next_f[A];
  const auto load = [&](int i) {
#pragma unroll
    for (int x = 0; x < A; ++x) {
      next[x] = to[min(i + x, n - 2) * up];
      next_f[x] = kept[static_cast<int64_t>(min(i + x, n - 2)) * a.hv];
    }
  };
  load(0);
  for (int i = 0; i < n; i += A) {
#pragma unroll
    for (int x = 0; x < A; ++x) {
      added[x] = next[x];
      f[x] = next_f[x];
    }
    if (i + A < n) load(i + A);
#pragma unroll
    for (int x = 0; x < A; ++x) {
      if (i + x >= n) return;
      to[(i + x) * up] = z;
      z = z * f[x] + added[x];
    }
  }
}

struct LinearSizes {
  int32_t tokens;  // a tile's
  int64_t tiles, slots;  // to launch, and there is room for as many as no smaller call has more of:
  int64_t most_tiles, most_slots;
  size_t kept, states, bytes;  // offsets, and all of it
};

// A tile's length. Under GDN_PREFILL_SEGMENTS it depends on the layer alone. Else the call's tokens set it: 2 chunks
// (the adding pass, whose work a longer tile would not lessen, then has the most workgroups), doubled until one head's work for a
// workgroup of 4 waves comes to about two workgroups a CU, where more would wait for a place; and until the scan's
// steps, one a tile, are few beside a tile's own. Calls, us, against the layer's own 8 chunks and whole sequences (32 heads,
// d = 128, bf16): 1024 tokens 41 (74, 93), 4096 87 (83, 347), the pack of 15717 tokens 233 (250, 696), 16 sequences of 1024 181
// (238, 161), 64 of them 636 (905, 623), one of 16384 among 31 of 256 417 (369, 1423). The rule knows the sum of the lengths alone:
// where many sequences of one length fill the card by themselves, WHOLE is the better choice by 2 to 13%. Half the tiles of the last rule (32 heads): 64 sequences 592, one of 16384
// among 31 of 256 354 (407); 8 heads, d = 64, one of 16384 tokens without the scan's rule 60 (49).
LinearSizes sizes(int32_t hv, int32_t d, int32_t n, int32_t total, int32_t form) {
  LinearSizes z{};
  const int64_t seqs = n < total ? n : total;
  int64_t whole = 0, most = 0;  // tiles' lengths that all tokens hold
  z.tokens = INT32_MAX;
  if (form != GDN_PREFILL_WHOLE) {
    const bool fixed = form == GDN_PREFILL_SEGMENTS;
    const int32_t chunks = fixed ? hv * d / 512 : 2, shortest = kChunk * (chunks < 2 ? 2 : chunks > 8 ? 8 : chunks);
    const int64_t cap = fixed ? INT32_MAX : 1 + 512 * 128 / (hv * d);
    int64_t tokens = shortest;
    const auto scan_heavy = [&] { return 16 * (tokens / kChunk) * (tokens / kChunk) < total / kChunk; };
    while (tokens * cap < total || (!fixed && scan_heavy())) tokens *= 2;
    if (total > kUncut && total > tokens) {
      z.tokens = static_cast<int32_t>(tokens);
      whole = total / tokens;
    }
    most = total / shortest < cap ? total / shortest : cap;
  }
  // a sequence of several tiles is longer than one: at most twice the whole tiles of all tokens
  const auto rooms = [&](int64_t w) { return w < seqs ? 2 * w : w + seqs; };
  z.tiles = seqs + whole;
  z.slots = rooms(whole);
  z.most_tiles = seqs + most;
  z.most_slots = rooms(most);
  const auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  z.kept = n > kWave ? up((z.most_tiles + z.most_slots) * sizeof(Place)) : 0;
  z.states = z.kept + up(z.most_slots * hv * sizeof(float));
  z.bytes = z.states + z.most_slots * hv * static_cast<size_t>(d) * d * sizeof(float);
  return z;
}

template <int D, typename T>
hipError_t prefill_dt(const LinearArgs& a, LinearPlan p, const LinearSizes& z, hipStream_t s) {
  // fewer than 2^31 threads a launch
  const int64_t most = ((int64_t)1 << 31) / (static_cast<int64_t>(a.hv) * (D * D / 4 > 512 ? D * D / 4 : 512));
  hipError_t e = hipSuccess;
  const auto in_turns = [&](int64_t n, auto launch) {
    for (int64_t f = 0; f < n && e == hipSuccess; f += most) {
      p.first = static_cast<int32_t>(f);
      launch(static_cast<unsigned>((n - f < most ? n - f : most) * a.hv));
      e = hipGetLastError();
    }
  };
  in_turns(z.slots, [&](unsigned grid) {
    linear_chunks_kernel<D, T, float, false><<<grid, LinearCfg<D, T, false>::THREADS, 0, s>>>(a, p);
  });
  in_turns(z.slots, [&](unsigned grid) { linear_scan_kernel<D><<<grid * (D * D / 4 / kScanThreads), kScanThreads, 0, s>>>(a, p); });
  in_turns(z.tiles, [&](unsigned grid) {
    constexpr int threads = LinearCfg<D, T, true>::THREADS;
    if (a.o_bf16) linear_chunks_kernel<D, T, uint16_t, true><<<grid, threads, 0, s>>>(a, p);
    else linear_chunks_kernel<D, T, float, true><<<grid, threads, 0, s>>>(a, p);
  });
  return e;
}

template <typename T>
hipError_t prefill_t(const LinearArgs& a, const LinearPlan& p, const LinearSizes& z, hipStream_t s) {
  switch (a.d) {
    case 32: return prefill_dt<32, T>(a, p, z, s);
    case 64: return prefill_dt<64, T>(a, p, z, s);
    default: return prefill_dt<128, T>(a, p, z, s);
  }
}

}  // namespace

hipError_t launch_linear_decode(const LinearArgs& a, int32_t m, hipStream_t s) {
  return a.bf16 ? decode_t<uint16_t>(a, m, s) : decode_t<float>(a, m, s);
}

size_t linear_workspace_bytes(int32_t hv, int32_t d, int32_t num_seqs, int32_t total_tokens, int32_t form) {
  return sizes(hv, d, num_seqs, total_tokens, form).bytes;
}

hipError_t launch_linear_prefill(const LinearArgs& a, const int32_t* cu, int32_t n, int32_t total, void* workspace, hipStream_t s) {
  const LinearSizes z = sizes(a.hv, a.d, n, total, a.form);
  char* ws = static_cast<char*>(workspace);
  LinearPlan p{cu, n, total, z.tokens, nullptr, nullptr, reinterpret_cast<float*>(ws + z.states),
               reinterpret_cast<float*>(ws + z.kept), 0};
  if (n > kWave) {
    Place* tiles = reinterpret_cast<Place*>(ws);
    Place* slots = tiles + z.tiles;
    linear_table_kernel<<<1, kTableThreads, 0, s>>>(p, tiles, static_cast<int>(z.tiles), slots, static_cast<int>(z.slots));
    if (const hipError_t e = hipGetLastError()) return e;
    p.tiles = tiles;
    p.slots = slots;
  }
  return a.bf16 ? prefill_t<uint16_t>(a, p, z, s) : prefill_t<float>(a, p, z, s);
}

}  // namespace gdn
