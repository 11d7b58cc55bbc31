// Speculative decoding over the slot pool, gfx950: a tree of drafted tokens per slot answered
// against the slot's state (tree_verify_kernel), and the slot moved along the accepted root path
// (tree_accept_kernel). include/gdn.h, gdn_tree_verify and gdn_tree_accept, has the formulas.
// (The layer's decode branch, "System Design" (project_6), "GDN Kernel Dispatch Detail", for
// every node of a tree; slots addressed as in aprender #5279, "Phase plan", phase P5.)

#include "conv_taps.h"
#include "device_common.h"
#include "launch.h"
#include "mma.h"

namespace gdn {
namespace {

typedef __attribute__((address_space(1))) f32x4 gf32x4;
typedef __attribute__((address_space(1))) float gfloat;
typedef __attribute__((address_space(4))) const uint64_t cu64;
typedef __attribute__((address_space(4))) const int32_t ci32;

// An element of an input (bf16 bits or fp32) as fp32.
template <typename T>
__device__ __forceinline__ float elem_f32(T v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
  else return v;
}

// e^x for x <= 0, a decay: 2^(x log2 e) on the hardware's base-2 exponential. The rounding of the
// exponent is off by |x| 2^-24 of the result, at most 0.37 x 2^-24 of 1 for any x.
__device__ __forceinline__ float decay(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// A sum of g over a path in two halves, so that the difference of two of them keeps the digits of the mild
// tokens behind a strongly forgetting one. A g below -128 counts as -128: e^-128 is 0 in fp32 as well, and
// the sums of 64 nodes stay above -8192, whose halves are good to 2^-35.
constexpr float kForget = -128.0f;
struct Gamma {
  float hi, lo;
};
__device__ __forceinline__ Gamma gamma_of(float g) { return Gamma{g < kForget ? kForget : g, 0.f}; }  // (a NaN stays)
__device__ __forceinline__ Gamma operator+(const Gamma& a, const Gamma& b) {
  const float s = a.hi + b.hi, bb = s - a.hi;
  const float lo = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
  const float hi = s + lo;
  return Gamma{hi, lo - (hi - s)};
}

// Slot i's rows: the first, and how many the call works on (none where cu_nodes does not lie
// inside [0, total]).
__device__ __forceinline__ void tree_span(const int32_t* cu, int i, int total, int max_nodes, int& first, int& n) {
  const int b = ((ci32*)cu)[i], e = ((ci32*)cu)[i + 1];
  const int len = e - b < max_nodes ? e - b : max_nodes;
  first = b;
  n = b < 0 || e <= b || b >= total ? 0 : len < total - b ? len : total - b;
}

// Node t's parent inside its tree (-1: the slot itself).
__device__ __forceinline__ int parent_of(const int32_t* parents, int first, int t) {
  if (t < 0) return -1;
  if (!parents) return t - 1;
  const int p = parents[first + t];
  return p >= -1 && p < t ? p : -1;
}

// The record's G holds one fp32 number, whose steps grow with it. So where a parent's is below -128 and the
// node's own g above that, the sum starts again from the node: G = g. Such a parent is at the end of a
// path whose sum of g is below -128, and no other node's G behind it rises above its parent's, which is how the
// reader knows. Lane t: sum = the path's sum (used while above -128), g and parent of node t. In two halves here
// as well, so that an entry is rounded once and not once a node of its path.
__device__ __forceinline__ float restarted_sum(Gamma sum, float g, int par, int n) {
  Gamma rec = sum;
  for (int s = 0; s < n; ++s) {  // (after s rounds right down to depth s)
    const Gamma above = {__shfl(rec.hi, par >= 0 ? par : 0), __shfl(rec.lo, par >= 0 ? par : 0)};
    const bool past = par >= 0 && above.hi < kForget;
    if (past || sum.hi <= kForget) {
      rec = par < 0 || (past && g > above.hi) ? Gamma{g, 0.f} : above + Gamma{g, 0.f};
      if (!(fabsf(rec.lo) < __builtin_inff())) rec.lo = 0.f, rec.hi = above.hi + g;  // (a sum beyond fp32's range)
    }
  }
  return rec.hi;
}

// Renumbers grid.x so that consecutive k-heads, which read and write neighbouring bytes, share an
// XCD's L2 (see decode.hip).
__device__ __forceinline__ int xcd_head() {
  const int n = gridDim.x, b = blockIdx.x;
  return (n % 8 == 0) ? (b % 8) * (n / 8) + b / 8 : b;
}

// The products with d terms, in the two policies of gdn_mma. FP32: v_mfma_f32_16x16x4_f32.
// BF16X3, for inputs of 8 significant bits: fp16 operands that carry an fp32 value in two halves: hi = fp16(x),
// lo = fp16(x - hi), about 22 significant bits. A product is hi hi' + hi lo' + lo hi' on
// v_mfma_f32_16x16x32_f16 with fp32 accumulation; what is left out is 2^-22 of it at most, typically 2^-24, as
// an fp32 product's own rounding. fp16 has little range, so every row is first multiplied by a power of two
// (exact) that puts its norm (or largest value) at 2^12 .. 2^13, and the result by its inverse. A value far
// below its row's norm is so held to 2^-37 of the norm, not to 2^-22 of itself: what a sum loses is small beside
// the rows' norms, but not always beside the sum, which is why fp32 inputs do not take this form by default.
// 64 slots x 64 nodes of bf16 x take 121 us with pairs and 162 us in fp32, x 16 nodes 44 and 48 us.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

struct Half2 {
  f16x8 hi, lo;
};

struct PairMma {
  static constexpr bool kFull = false;
  static constexpr int kStep = 32;
  typedef Half2 Frag;
  __device__ __forceinline__ static void mma(f32x4& acc, const Frag& a, const Frag& b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.lo, b.hi, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.lo, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.hi, acc, 0, 0, 0);
  }
  __device__ __forceinline__ static void mma3(f32x4 (&acc)[3], const Frag& a, const Frag& b) {
    acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.hi, acc[0], 0, 0, 0);
    acc[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.lo, b.hi, acc[1], 0, 0, 0);
    acc[2] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.hi, b.lo, acc[2], 0, 0, 0);
  }
};

// (The steps' LDS reads are fenced in twos where two workgroups share a CU: all of them ahead of the products
// spill, 64 slots x 16 nodes of fp32 x 51 -> 67 us.)
struct FullMma {
  static constexpr bool kFull = true;
  static constexpr int kStep = 16;
  typedef f32x4 Frag;
  __device__ __forceinline__ static void mma(f32x4& acc, const Frag& a, const Frag& b) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[q], b[q], acc, 0, 0, 0);
  }
  // ... on three independent chains (summed by total())
  __device__ __forceinline__ static void mma3(f32x4 (&acc)[3], const Frag& a, const Frag& b) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q % 3] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[q], b[q], acc[q % 3], 0, 0, 0);
  }
};

// The exponent that takes a magnitude below 2^e to below 2^13 (kept where its inverse is finite too).
__device__ __forceinline__ int f16_shift(int e) { return e < -97 ? 110 : 13 - e; }

// x * mul, mul a power of two, in two halves, one instruction a half: fp16(x mul + 0) and
// fp16(x mul - hi). (With any other factor the first would be rounded once in this form and twice as a
// product and a conversion, and the compiler takes either.)
__device__ __forceinline__ _Float16 half_hi(float x, float mul) { return static_cast<_Float16>(fmaf(x, mul, 0.0f)); }
__device__ __forceinline__ _Float16 half_lo(float x, float mul, _Float16 hi) {
  return static_cast<_Float16>(fmaf(x, mul, -static_cast<float>(hi)));
}

// (where the magnitudes' sum overflows: false as well)
__device__ __forceinline__ bool all_finite(const f32x4& v) {
  return (fabsf(v[0]) + fabsf(v[1])) + (fabsf(v[2]) + fabsf(v[3])) < __builtin_inff();
}

// v of the lane 16 (or 32) away combined with the lane's own by op.
template <typename F>
__device__ __forceinline__ float across16(float v, F op) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
template <typename F>
__device__ __forceinline__ float across32(float v, F op) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return op(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// left * right + acc for 16x16 fp32 tiles: left given as MFMA's left operand (lane l: row l % 16, columns
// 4 (l / 16) + q), right and acc as results (rows 4 (l / 16) + q of column l % 16). The left operand of
// a matrix is the result layout of its transpose.
__device__ __forceinline__ f32x4 mul16(const f32x4& left, const f32x4& right, f32x4 acc) {
#pragma unroll
  for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(left[q], right[q], acc, 0, 0, 0);
  return acc;
}

// (I - A)^-1 of a strictly lower triangular 16x16 tile A (result layout in and out). With D the inverses
// of I - A's 4x4 diagonal blocks, formed by substitution inside the four lanes that hold a block, L the
// rest of A and X = D L (X^4 = 0):  (I - A)^-1 = (I + X^2)(D + X D).
// Five products in three dependent steps; sixteen steps of substitution took two to three times as long.
__device__ __forceinline__ f32x4 unit_lower_inverse(const f32x4& a, int lane) {
  const int c4 = lane / 16, k = lane % 4;
  const bool on_diagonal = (lane % 16) / 4 == c4;
  // entries of the lane's 4x4 diagonal block: column c from lane c of the quad (quad_perm [c c c c])
  const float a10 = dpp_f32<0x00>(a[1]), a20 = dpp_f32<0x00>(a[2]), a30 = dpp_f32<0x00>(a[3]);
  const float a21 = dpp_f32<0x55>(a[2]), a31 = dpp_f32<0x55>(a[3]), a32 = dpp_f32<0xAA>(a[3]);
  const float d20 = fmaf(a21, a10, a20), d31 = fmaf(a32, a21, a31);
  const float d30 = fmaf(a32, d20, fmaf(a31, a10, a30));
  const float z = 0.f, one = on_diagonal ? 1.f : 0.f;
  const auto pick = [&](float v0, float v1, float v2, float v3) {
    const float v = k == 0 ? v0 : k == 1 ? v1 : k == 2 ? v2 : v3;
    return on_diagonal ? v : 0.f;
  };
  // D's column k (result layout) and row k (left operand)
  const f32x4 d = {k == 0 ? one : z, pick(a10, 1.f, z, z), pick(d20, a21, 1.f, z), pick(d30, d31, a32, 1.f)};
  const f32x4 dl = {pick(1.f, a10, d20, d30), pick(z, 1.f, a21, d31), pick(z, z, 1.f, a32), k == 3 ? one : z};
  f32x4 rest;
#pragma unroll
  for (int q = 0; q < 4; ++q) rest[q] = on_diagonal ? 0.f : a[q];
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const f32x4 x = mul16(dl, rest, zero);   // X = D L
  const f32x4 xt = mul16(rest, dl, zero);  // X^T = L^T D^T (L's result layout is L^T's left operand, D^T's right is dl)
  const f32x4 sqt = mul16(x, xt, zero);    // (X^2)^T = X^T X^T
  const f32x4 y = mul16(xt, d, d);         // D + X D
  return mul16(sqt, y, y);
}

// The same where a path's products overflow: lane c < 16 substitutes for column c, over the entries that are
// not zero alone, so that an infinity stays on the path it belongs to. a: room for the tile, rows of `stride`.
// (A call of its own: inlined, its loops cost the kernels registers, 64 slots x 16 nodes of fp32 x 45 -> 51 us.)
__device__ __attribute__((noinline)) void careful_inverse(f32x4 tile, float* a, int stride, float (*t)[20], int lane) {
#pragma unroll
  for (int q = 0; q < 4; ++q) a[(4 * (lane / 16) + q) * stride + lane % 16] = tile[q];
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  if (lane >= 16) return;
  for (int i = 0; i < 16; ++i) {
    float x = i == lane ? 1.f : 0.f;
    for (int k = 0; k < i; ++k) {
      const float v = a[i * stride + k];
      if (v != 0.f) x = fmaf(v, t[k][lane], x);
    }
    t[i][lane] = x;
  }
}

__device__ __forceinline__ void barrier_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// One workgroup per slot and up to HP v-heads of one k-head, so that they share its q and k; one wave
// per 16 state rows of a head. PAR heads run side by side on waves of their own, the others after them
// on the same waves (their state rows are loaded while the head before finishes). NB = blocks of 16 nodes.
//
// The rows of the state do not mix, so with K, Q [N][d] the normalised tokens and S the wave's 16
// rows everything is small matrix products on 16x16 tiles:
//   M = K S^T, W = Q S^T               [N][16]
//   A_ij = -beta_i e^(G_i - G_j) k_i.k_j for j above i, else 0;   P_ij = e^(G_i - G_j) q_i.k_j, j above or at i
//   U = (I - A)^-1 (beta (V - e^G M)), O = e^G W + P U
// (I - A) is unit lower triangular (parents come first): its 16x16 diagonal blocks are inverted by five
// products (unit_lower_inverse), the rest is block substitution. The products with d terms (M, W, A, P) run in the call's
// policy (MMA), the others on fp32 MFMA with the contraction index dealt as 4 (l / 16) + r, so that a result
// tile (lane l: rows 4 (l / 16) + r of column l % 16) is the right operand of the next product as it stands.
//
// Everything a workgroup reads from memory is loaded before anything is computed: its state rows
// (registers), the x rows of its nodes and the conv-state rows before them (LDS, as they came; the conv
// then gathers each node's window there), parents, g and beta. The barriers order LDS only, so the state
// rows stay in flight across them.
//
// What bounds it. At 16/32 heads, d = 128, bf16, 64 slots read 134 MB of states: 16-node trees take 42 us (182 MB
// in all, 4.3 TB/s), 64-node trees 121 to 126 us (290 MB and 8.6 GFLOP, of which the products with d terms are
// issued three times). HBM is busy at its streaming rate while the workgroups of a round load, and mostly idle
// while they compute: the two workgroups that a CU holds (one, for the largest trees: of its 157 KB of LDS
// the two heads' A, P and inverses take 80, K and Q 74) start together and stay in step. Neither the
// vector units (36% of the time) nor MFMA (14%; 23% for the largest trees) is the limit there, LDS
// fragment reads and the substitution's dependent products are.
// A workgroup that took several items in turn and loaded the next one's state and x during the
// substitution needed 130 to 300 bytes of spilled registers a lane. One slot with 4 nodes takes 8.4 us, a chain
// of about 17k cycles: two dependent memory round trips, the conv, A's diagonal blocks, M and W, the substitution.
// Part of it is work that a single head does not need: v's conv runs for two heads, whether or not there is a second.
//
// A zero of A or P times an infinity or a NaN would carry a broken token into branches that do not
// see it. So such values never enter the products: a k that is not finite marks its node, a row of A that is
// not (g or beta) marks its node for that head, a right side beta (v - e^G M) - .. or a u that is not marks it for that
// state row, zeros go in their place, and the results of the marked nodes and their descendants are set to
// NaN at the end. An inverse that is not finite (a path of unnormalised keys that diverges) is formed
// again without products by zeros; its rows are then not finite on that path alone, and so u's.

// q and k in LDS: fp32 rows, or hi and lo rows of halves (inside a row see place()).
template <typename MMA, int N, int D>
struct QkRows {
  static constexpr int S = D + 16;  // fp16 values of a row (conflict-free fragment reads)
  _Float16 v[2][2][N][S];           // q, k; hi, lo
};
template <int N, int D>
struct QkRows<FullMma, N, D> {
  static constexpr int S = D + 4;
  float v[2][N][S];
};

template <typename MMA, typename T, int K, int D, int NB, int HP>
struct VerifyLds {
  static constexpr int N = 16 * NB;
  static constexpr int PS = N + 4;   // floats of a row of A and P
  static constexpr int XS = 2 * D + 16 / sizeof(T);  // values of a row of x's q and k channels
  static constexpr int VS = HP * D + 16 / sizeof(T);  // ... and of the heads' v channels
  struct Products {
    float a[N][PS];       // A (its diagonal blocks stay in registers)
    float p[N][PS];       // P
    float t[NB][16][20];  // inverses of the diagonal blocks
  };
  // rows of x: the conv-state rows, oldest first, then the nodes'
  union {
    T x[K - 1 + N][XS];
    Products m[HP];  // (written once the conv is done with x)
  };
  union {
    T xv[K - 1 + N][VS];
    QkRows<MMA, N, D> qk_shared[NB > 1 ? 1 : 0];  // (larger trees: written once v is convolved)
  };
  QkRows<MMA, N, D> qk_own[NB > 1 ? 0 : 1];
  __device__ __forceinline__ auto& qk() { return (NB > 1 ? qk_shared : qk_own)[0].v; }
  alignas(16) float inv[2][N];  // pairs: inverse of the row's power of two, q and k
  alignas(16) float gam[HP][N], gam_lo[HP][N], eg[HP][N], beta[HP][N];
  uint32_t anc[N][2];         // ancestors (bit j: node j), not itself
  uint32_t kbad[2], qbad[2];  // nodes whose k (q) is not finite
  uint32_t abad[HP][2];       // nodes whose row of A is not finite, by head
};

// Where value k of a row of q or k lies in LDS: a lane's 8 values of a 32-wide MFMA step are adjacent. The
// step's contraction index is dealt to the lane group c = l / 16 as {4 c + 0..3, 16 + 4 c + 0..3}, the
// columns that two 16-byte state loads bring.
__device__ __forceinline__ constexpr int place(int k) {
  return (k / 32) * 32 + ((k % 16) / 4) * 8 + ((k % 32) / 16) * 4 + k % 4;
}

// Heads of a workgroup (HP) and how many of them side by side on waves of their own (PAR), the rest one after
// the other. Side by side is for the smaller head dims' larger trees, whose four or two waves a head would convolve
// the tokens alone: 64 slots x 64 nodes take 65 us against 107 (d = 32), 66 against 97 (d = 64, bf16 x) and 81 against
// 107 (fp32 x), one slot 15 to 17 against 18 to 21.
// JOIN, the heads that a wave takes together, is 1. Two spare LDS reads at 64 more registers, and lose everywhere:
// 64 slots x 64 nodes of d = 128 take 121 us one after the other and 124 together (fp32 products 161 and 169), one
// slot 21.5 and 22.9. The loops over it stay all the same: without them the compiler lays the blocks out so that
// the larger trees spill (129 us, fp32 products 247).
constexpr int kVerifyHeads = 2;
constexpr int verify_par(int nb, int d) { return nb > 2 && d < 128 ? 2 : 1; }

template <typename MMA, typename T, int K, int D, int NB, int SILU>  // (SILU -1: as the arguments say)
__global__ __launch_bounds__(D * 4 * verify_par(NB, D), (D < 128 ? 1 : NB <= 2 ? 4 : 2)) void tree_verify_kernel(
    TreeArgs a, int32_t heads, int32_t chunks) {
  constexpr int HP = kVerifyHeads, PAR = verify_par(NB, D), SEQ = HP / PAR, JOIN = 1;
  using Lds = VerifyLds<MMA, T, K, D, NB, HP>;
  const bool silu_on = SILU < 0 ? a.silu != 0 : SILU != 0;
  constexpr int WH = D / 16;         // waves of a head
  constexpr int W = WH * PAR;        // waves
  constexpr int NT = W * kWave;      // threads
  constexpr int N = 16 * NB;
  constexpr int CH = 2 * D / 4;      // 4-channel pieces of a node's q and k channels
  using Raw = typename Vec8<T>::Raw;
  using V4 = Vec4<T>;
  __shared__ __attribute__((aligned(16))) Lds lds;

  const RecurArgs& r = a.r;
  const int i = blockIdx.y;
  const uint64_t sp = ((cu64*)r.state_ptrs)[i];
  const uint64_t cp = ((cu64*)a.conv_ptrs)[i];
  int first, n;
  tree_span(a.cu_nodes, i, a.total_nodes, a.max_nodes, first, n);
  if (n == 0 || sp == 0 || cp == 0) return;  // (the whole workgroup)
  // the workgroup's v-heads: j0 .. j0 + nh - 1 of k-head h
  const int bx = xcd_head();
  const int h = chunks == 1 ? bx : bx / chunks;
  const int g0 = (bx - h * chunks) * heads;
  const int j0 = h * r.group + g0;
  const int nh = heads < r.group - g0 ? heads : r.group - g0;
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int hw = PAR == 1 ? 0 : w / WH;   // the wave's first head (of the workgroup's)
  const int row_w = (w % WH) * 16;        // and its state rows
  const int c4 = lane / 16, l16 = lane % 16;
  const int C = a.channels;

  // every wave: lane t's parent (the root for lanes past the tree)
  const int par = lane < n ? parent_of(a.parents, first, lane) : -1;
  // wave t < nh: g and beta of head t
  const bool tree_wave = w < nh;
  const int64_t gi = static_cast<int64_t>(first + lane) * r.hv + j0 + w;
  const float gval = tree_wave && lane < n ? r.g[gi] : 0.f;
  const float bval = tree_wave && lane < n ? r.beta[gi] : 0.f;
  // x and conv-state rows, on their way to LDS
  const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(first) * a.x_stride;
  const T* cs = reinterpret_cast<const T*>(cp);
  constexpr int LX = (2 + HP) * D / 8;     // lanes on one row
  constexpr int RW = W * kWave / LX;       // rows a pass
  constexpr int IT = (K - 1 + N + RW - 1) / RW;
  const int px = (lane % LX) * 8;          // the lane's channels within q | k | the heads' v
  const int pn = (2 + nh) * D;
  const int rx = w * (kWave / LX) + (kWave == LX ? 0 : lane / LX);
  const int chx = px < D ? h * D + px : px < 2 * D ? (r.hk - 1 + h) * D + px : (2 * r.hk - 2 + j0) * D + px;
  Raw raw[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int row = it * RW + rx;
    if (row < K - 1 + n && px < pn)
      raw[it] = Vec8<T>::load_raw((row < K - 1 ? cs + static_cast<int64_t>(row) * C : x + (row - (K - 1)) * a.x_stride) + chx);
  }
  // taps of the lane's v channels (one a head), and of the thread's 4 q or k channels
  T vtap[SEQ][K], vbias[SEQ];
#pragma unroll
  for (int q = 0; q < SEQ; ++q) {
    const int lh = q * PAR + hw < nh ? q * PAR + hw : 0;
    const int vch = (2 * r.hk + j0 + lh) * D + row_w + l16;
#pragma unroll
    for (int t = 0; t < K; ++t) vtap[q][t] = static_cast<const T*>(a.w)[static_cast<int64_t>(vch) * K + t];
    vbias[q] = static_cast<const T*>(a.b ? a.b : a.w)[vch];  // (taps stand in when there is no bias)
  }
  const int piece = tid % CH;
  const bool is_k = piece * 4 >= D;
  const int d0 = (piece * 4) % D;
  const int ch0 = (is_k ? r.hk * D : 0) + h * D + d0;
  typename V4::Raw tap[K], bias;
  const auto load_taps = [&]() {
#pragma unroll
    for (int t = 0; t < K; ++t) tap[t] = V4::load_raw(static_cast<const T*>(a.w) + static_cast<int64_t>(ch0) * K + 4 * t);
    bias = V4::load_raw(static_cast<const T*>(a.b ? a.b : a.w) + ch0);
  };
  // (fp32 rows of up to 32 nodes, their taps and the state do not fit two workgroups' registers together:
  // 64 slots x 32 nodes take 78 us (pairs 61) with the taps' loads behind the rows', 89 us (66) with all of them
  // here, spilled)
  constexpr bool kLateTaps = sizeof(T) == 4 && NB == 2 && D == 128;
  if constexpr (!kLateTaps) load_taps();
  // the wave's state rows of its head lh: lane (c4, l16) holds columns 16 e + 4 c4 .. + 3 of row l16
  f32x4 s[JOIN][D / 16];
  const auto load_state = [&](f32x4 (&s)[D / 16], int lh) {
    const gf32x4* S = (const gf32x4*)(reinterpret_cast<const float*>(sp) +
                                      (static_cast<int64_t>(j0 + lh) * D + row_w + l16) * D);
#pragma unroll
    for (int e = 0; e < D / 16; ++e) s[e] = __builtin_nontemporal_load(S + 4 * e + c4);
  };
#pragma unroll
  for (int t = 0; t < JOIN; ++t) {
    if (t * PAR + hw < nh) load_state(s[t], t * PAR + hw);
  }
  __builtin_amdgcn_sched_barrier(0);  // every load above is issued before the first wait
  if (tid < 2) {
    lds.kbad[tid] = lds.qbad[tid] = 0;
#pragma unroll
    for (int t = 0; t < HP; ++t) lds.abad[t][tid] = 0;
  }
  // lane t: the LDS rows of the K-1 rows before node t, 8 bits each, the nearest one lowest
  int back = 0;
  {
    int at = lane + K - 1;
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      const int up = __shfl(par, at >= K - 1 ? at - (K - 1) : 0);
      at = at >= K - 1 ? K - 1 + up : at - 1;  // (parent -1 is row K-2, the newest conv-state row)
      back |= at << (8 * t);
    }
  }
  if (tree_wave) {
    // ancestors and sums of g along the root path by doubling: after round s they cover 2^s levels
    int up = par;
    Gamma gam = gamma_of(gval);
    uint32_t lo = up >= 0 && up < 32 ? 1u << up : 0u, hi = 0u;
    if constexpr (N > 32) hi = up >= 32 ? 1u << (up - 32) : 0u;
    while (__any(up >= 0)) {
      const int from = up >= 0 ? up : lane;
      const uint32_t lo2 = __shfl(lo, from), hi2 = N > 32 ? __shfl(hi, from) : 0u;
      const Gamma g2 = {__shfl(gam.hi, from), __shfl(gam.lo, from)};
      const int up2 = __shfl(up, from);
      if (up >= 0) {
        lo |= lo2;
        hi |= hi2;
        gam = gam + g2;
        up = up2;
      }
    }
    float rec = gam.hi;
    if (a.gamma_rec && __any(gam.hi <= kForget)) rec = restarted_sum(gam, gval, par, n);
    if (lane < N) {
      if (w == 0) {
        lds.anc[lane][0] = lo;
        lds.anc[lane][1] = hi;
      }
      lds.gam[w][lane] = gam.hi;
      lds.gam_lo[w][lane] = gam.lo;
      lds.eg[w][lane] = expf(gam.hi) * (1.0f + gam.lo);
      lds.beta[w][lane] = bval;
      if (lane < n && a.gamma_rec) a.gamma_rec[gi] = rec;
    }
  }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int row = it * RW + rx;
    if (row < K - 1 + n && px < pn) *reinterpret_cast<Raw*>(px < 2 * D ? &lds.x[row][px] : &lds.xv[row][px - 2 * D]) = raw[it];
  }
  if constexpr (kLateTaps) load_taps();

  barrier_lds();

  // v of the lane's nodes (4 c4 + 0..3 of every block) at its state row, a head after the other
  float v[SEQ][NB][4];
  const auto conv_v = [&]() {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (16 * b >= n) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * b + 4 * c4 + e;
        const int rows = __shfl(back, t);
#pragma unroll
        for (int sq = 0; sq < SEQ; ++sq) {
          const int off = (sq * PAR + hw) * D + row_w + l16;
          float acc = a.b ? elem_f32<T>(vbias[sq]) : 0.f;
#pragma unroll
          for (int q = 0; q < K - 1; ++q)
            acc = fmaf(elem_f32<T>(vtap[sq][q]), elem_f32<T>(lds.xv[(rows >> (8 * (K - 2 - q))) & 255][off]), acc);
          acc = fmaf(elem_f32<T>(vtap[sq][K - 1]), elem_f32<T>(lds.xv[K - 1 + t][off]), acc);
          v[sq][b][e] = silu_on ? silu(acc) : acc;  // (rows past the tree hold anything)
        }
      }
    }
  };
  if constexpr (NB > 1) {
    conv_v();
    barrier_lds();
  }
  // q and k: a thread convolves 4 channels (always the same ones) of one node a pass
#pragma unroll
  for (int pass = 0; pass < N / (NT / CH); ++pass) {
    if (pass * (NT / CH) >= n) break;
    const int t = pass * (NT / CH) + tid / CH;
    const int rows = __shfl(back, t);
    const int off = (is_k ? D : 0) + d0;
    typename V4::Raw win[K - 1];
#pragma unroll
    for (int q = 0; q < K - 1; ++q) win[q] = V4::load_raw(&lds.x[(rows >> (8 * (K - 2 - q))) & 255][off]);
    float y[4];
    conv4_raw<T, K>(tap, bias, a.b != nullptr, win, V4::load_raw(&lds.x[K - 1 + t][off]), silu_on, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = t < n ? y[e] : 0.f;  // (rows past the tree hold anything)
    const auto row_sum = [](float z) {  // over the D / 4 lanes of a row
      z = group_sum<(D / 4 < 16 ? D / 4 : 16)>(z);
      if constexpr (D / 4 > 16) z = across16(z, [](float p, float q) { return p + q; });
      return z;
    };
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) ss = fmaf(y[e], y[e], ss);
    ss = row_sum(ss);
    float f = r.qk_norm && t < n ? __builtin_amdgcn_rsqf(ss + r.eps) : 1.0f;
    if (!is_k) f *= r.scale;
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[e] = y[e] * f;
      asm("" : "+v"(z[e]));  // (rounded here, whatever becomes of it)
    }
    if (t < n && is_k && a.k_rec && g0 == 0)
      *reinterpret_cast<f32x4*>(a.k_rec + (static_cast<int64_t>(first + t) * r.hk + h) * D + d0) =
          f32x4{z[0], z[1], z[2], z[3]};
    // |row| < 2^((e + 1) / 2), from the sum of squares where that is far inside the fp32 range
    const float norm2 = ss * f * f;
    int top = (__builtin_amdgcn_frexp_expf(norm2) + 1) >> 1;
    if (!(norm2 > 0x1p-100f && norm2 < 0x1p100f) && t < n) {  // (the row's threads agree on ss and f)
      // a row of zeros, of very large or small values, or with a value that is not finite: its largest
      if (row_sum((z[0] * 0.f + z[1] * 0.f) + (z[2] * 0.f + z[3] * 0.f)) != 0.f) {
        atomicOr(&(is_k ? lds.kbad : lds.qbad)[t >> 5], 1u << (t & 31));
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = 0.f;
      }
      float most = fmaxf(fmaxf(fabsf(z[0]), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3])));
#pragma unroll
      for (int m = 1; m < D / 4; m *= 2) most = fmaxf(most, __shfl_xor(most, m));
      top = __builtin_amdgcn_frexp_expf(most);
    }
    if constexpr (MMA::kFull) {
      *reinterpret_cast<f32x4*>(&lds.qk()[is_k][t][d0]) = f32x4{z[0], z[1], z[2], z[3]};
    } else {
      const int sh = f16_shift(top);
      if (d0 == 0) lds.inv[is_k][t] = ldexpf(1.0f, -sh);
      const float mul = ldexpf(1.0f, sh);
      f16x4 hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = half_hi(z[e], mul);
        lo[e] = half_lo(z[e], mul, hi[e]);
      }
      *reinterpret_cast<f16x4*>(&lds.qk()[is_k][0][t][place(d0)]) = hi;
      *reinterpret_cast<f16x4*>(&lds.qk()[is_k][1][t][place(d0)]) = lo;
    }
  }
  barrier_lds();

  const auto frag = [&](int which, int b, int step) -> typename MMA::Frag {
    if constexpr (MMA::kFull) {
      return *reinterpret_cast<const f32x4*>(&lds.qk()[which][16 * b + l16][step * 16 + c4 * 4]);
    } else {
      const int at = step * 32 + c4 * 8;
      return Half2{*reinterpret_cast<const f16x8*>(&lds.qk()[which][0][16 * b + l16][at]),
                   *reinterpret_cast<const f16x8*>(&lds.qk()[which][1][16 * b + l16][at])};
    }
  };
  // A and P of all heads: the lower blocks of k k^T and q k^T, dealt to the waves, k k^T's diagonal
  // blocks first; the wave that has one inverts I - A there, for all heads at once
  {
    constexpr int NL = NB * (NB + 1) / 2;
    for (int task = w; task < 2 * NL; task += W) {
      const bool is_p = task >= NL;
      int bi, bj;
      if (task < NB) {
        bi = bj = task;
      } else {  // the other blocks of A by rows, then P's
        int rest = is_p ? task - NL : task - NB;
        bi = is_p ? 0 : 1;
        while (rest >= (is_p ? bi + 1 : bi)) rest -= is_p ? ++bi : bi++;
        bj = rest;
      }
      if (16 * bi >= n) continue;
      const int col = 16 * bj + l16, row = 16 * bi + 4 * c4;
      f32x4 acc3[3];
      zero3(acc3);
#pragma unroll
      for (int e = 0; e < D / MMA::kStep; ++e) {
        MMA::mma3(acc3, frag(is_p ? 0 : 1, bi, e), frag(1, bj, e));
        if (MMA::kFull && NB <= 2 && e % 2) __builtin_amdgcn_sched_barrier(0);
      }
      bool use[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        use[q] = ((lds.anc[row + q][col >> 5] >> (col & 31)) & 1u) || (is_p && row + q == col);
      f32x4 acc = total(acc3);
      if constexpr (!MMA::kFull) acc = acc * *reinterpret_cast<const f32x4*>(&lds.inv[is_p ? 0 : 1][row]) * lds.inv[1][col];
      f32x4 tile[HP];
#pragma unroll
      for (int t = 0; t < HP; ++t) {
        tile[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (t >= nh) break;
        const float gcol = lds.gam[t][col], lcol = lds.gam_lo[t][col];
        const f32x4 grow = *reinterpret_cast<const f32x4*>(&lds.gam[t][row]);
        const f32x4 lrow = *reinterpret_cast<const f32x4*>(&lds.gam_lo[t][row]);
        const f32x4 brow = *reinterpret_cast<const f32x4*>(&lds.beta[t][row]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tile[t][q] =
              use[q] ? acc[q] * decay((grow[q] - gcol) + (lrow[q] - lcol)) * (is_p ? 1.0f : -brow[q]) : 0.f;
        // (a row of P reaches its own node's o alone)
        if (!is_p && __any(!all_finite(tile[t]))) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (!(fabsf(tile[t][q]) < __builtin_inff())) {
              atomicOr(&lds.abad[t][(row + q) >> 5], 1u << ((row + q) & 31));
              tile[t][q] = 0.f;
            }
        }
      }
      if (task < NB) {
#pragma unroll
        for (int t = 0; t < HP; ++t)
          if (t < nh) {
            const f32x4 x2 = unit_lower_inverse(tile[t], lane);
#pragma unroll
            for (int q = 0; q < 4; ++q) lds.m[t].t[bi][4 * c4 + q][l16] = x2[q];
            if (__any(!all_finite(x2))) careful_inverse(tile[t], &lds.m[t].a[16 * bi][16 * bi], Lds::PS, lds.m[t].t[bi], lane);
          }
      } else {
#pragma unroll
        for (int t = 0; t < HP; ++t)
          if (t < nh)
#pragma unroll
            for (int q = 0; q < 4; ++q) (is_p ? lds.m[t].p : lds.m[t].a)[row + q][col] = tile[t][q];
      }
    }
  }
  if constexpr (NB == 1) conv_v();
  const int64_t step = static_cast<int64_t>(r.hv) * D;  // values from a node's o (or u) to the next one's
#pragma unroll
  for (int sq = 0; sq < SEQ; sq += JOIN) {
    const auto head = [&](int t) { return (sq + t) * PAR + hw; };  // t < JOIN: the wave's heads of this round
    // M and W (the state rows as fp16 pairs)
    f32x4 m[JOIN][NB], o[JOIN][NB];
    float smul[JOIN], sinv[JOIN];  // pairs: the row's power of two and its inverse
    if (head(0) < nh) {
#pragma unroll
      for (int t = 0; t < JOIN; ++t) {
#pragma unroll
        for (int b = 0; b < NB; ++b) m[t][b] = o[t][b] = f32x4{0.f, 0.f, 0.f, 0.f};
        smul[t] = sinv[t] = 1.f;
        if constexpr (!MMA::kFull) {
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < D / 16; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) top = fmaxf(top, fabsf(s[t][e][q]));
          const auto larger = [](float p, float q) { return fmaxf(p, q); };
          top = across32(across16(top, larger), larger);
          const int sh = f16_shift(__builtin_amdgcn_frexp_expf(top));
          smul[t] = ldexpf(1.0f, sh);
          sinv[t] = ldexpf(1.0f, -sh);
        }
      }
#pragma unroll
      for (int e = 0; e < D / MMA::kStep; ++e) {
        typename MMA::Frag sf[JOIN];
#pragma unroll
        for (int t = 0; t < JOIN; ++t) {
          if constexpr (MMA::kFull) {
            sf[t] = s[t][e];
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float y = s[t][2 * e + q / 4][q % 4];
              sf[t].hi[q] = half_hi(y, smul[t]);
              sf[t].lo[q] = half_lo(y, smul[t], sf[t].hi[q]);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (16 * b < n) {
            const typename MMA::Frag kf = frag(1, b, e), qf = frag(0, b, e);
#pragma unroll
            for (int t = 0; t < JOIN; ++t) {
              MMA::mma(m[t][b], kf, sf[t]);
              MMA::mma(o[t][b], qf, sf[t]);
            }
          }
        if (MMA::kFull && NB <= 2 && e % 2) __builtin_amdgcn_sched_barrier(0);
      }
      if (head(1) < nh) load_state(s[0], head(1));
    }
    if (sq == 0) barrier_lds();  // A, P and the inverses of every head
    if (head(0) >= nh) break;
    // block substitution; u of block b replaces m[b]
    uint32_t bad[JOIN][2];  // marked nodes of the lane's state row
    const uint32_t qbad[2] = {lds.qbad[0], lds.qbad[1]};
    uint32_t marks = qbad[0] | qbad[1];
#pragma unroll
    for (int t = 0; t < JOIN; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bad[t][e] = lds.kbad[e] | (head(t) < nh ? lds.abad[head(t)][e] : 0u);
        marks |= bad[t][e];
      }
    bool dirty = marks != 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (16 * b >= n) break;
      const int t0 = 16 * b + 4 * c4;
      f32x4 kinv = {1.f, 1.f, 1.f, 1.f}, qinv = kinv;
      if constexpr (!MMA::kFull) {
        kinv = *reinterpret_cast<const f32x4*>(&lds.inv[1][t0]);
        qinv = *reinterpret_cast<const f32x4*>(&lds.inv[0][t0]);
      }
#pragma unroll
      for (int t = 0; t < JOIN; ++t) {
        const int lh = head(t);
        if (lh >= nh) break;
        const auto& mh = lds.m[lh];
        const f32x4 eg = *reinterpret_cast<const f32x4*>(&lds.eg[lh][t0]) * sinv[t];
        const f32x4 beta = *reinterpret_cast<const f32x4*>(&lds.beta[lh][t0]);
        f32x4 rhs;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          rhs[q] = t0 + q < n ? beta[q] * fmaf(-m[t][b][q], eg[q] * kinv[q], v[sq + t][b][q]) : 0.f;
          o[t][b][q] *= eg[q] * qinv[q];
        }
        const auto mark = [&](f32x4& v) {  // values that are not finite: zeros, their nodes marked
          if (!__any(!all_finite(v))) return;
          dirty = true;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint64_t off = __ballot(!(fabsf(v[q]) < __builtin_inff()));
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if ((off >> (16 * g + l16)) & 1u) bad[t][b / 2] |= 1u << (16 * (b % 2) + 4 * g + q);
            if ((off >> lane) & 1u) v[q] = 0.f;
          }
        };
#pragma unroll
        for (int b2 = 0; b2 < b; ++b2)
          rhs = mul16(*reinterpret_cast<const f32x4*>(&mh.a[16 * b + l16][16 * b2 + 4 * c4]), m[t][b2], rhs);
        mark(rhs);
        m[t][b] = mul16(*reinterpret_cast<const f32x4*>(&mh.t[b][l16][4 * c4]), rhs, f32x4{0.f, 0.f, 0.f, 0.f});
        mark(m[t][b]);
#pragma unroll
        for (int b2 = 0; b2 <= b; ++b2)
          o[t][b] = mul16(*reinterpret_cast<const f32x4*>(&mh.p[16 * b + l16][16 * b2 + 4 * c4]), m[t][b2], o[t][b]);
      }
    }
    // (stores after all of it: nothing the substitution waits for queues behind them)
#pragma unroll
    for (int t = 0; t < JOIN; ++t) {
      const int lh = head(t);
      if (lh >= nh) break;
      const int64_t base = static_cast<int64_t>(first + 4 * c4) * step + (j0 + lh) * D + row_w + l16;
      uint16_t* o16 = static_cast<uint16_t*>(r.o) + base;
      float* o32 = static_cast<float*>(r.o) + base;
      float* u32 = a.u_rec ? a.u_rec + base : nullptr;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (16 * b >= n) break;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int node = 16 * b + 4 * c4 + q;
          if (dirty) {
            const uint32_t self = 1u << (node & 31);
            const bool hit = (((lds.anc[node][0] | (node < 32 ? self : 0u)) & bad[t][0]) |
                              ((lds.anc[node][1] | (node < 32 ? 0u : self)) & bad[t][1])) != 0;
            if (hit) m[t][b][q] = __builtin_nanf("");
            if (hit || (qbad[node >> 5] & self)) o[t][b][q] = __builtin_nanf("");
          }
          if (node < n) {
            if (r.o_bf16)
              o16[(16 * b + q) * step] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[t][b][q]));
            else
              o32[(16 * b + q) * step] = o[t][b][q];
            if (u32) u32[(16 * b + q) * step] = m[t][b][q];
          }
        }
      }
    }
  }
}

template <typename T, int K, int D, int NB>
hipError_t verify_nb(const TreeArgs& a, int32_t m, hipStream_t s) {
  // Both heads of a pair on one workgroup once that leaves a workgroup for every CU. 16/32 heads of d = 128, trees of
  // 16 / 32 / 64 nodes, one head against two: 8 slots 10 / 14 / 26 us against 12 / 18 / 33, 16 slots (256 workgroups
  // of two) 15 / 22 / 48 against 13 / 20 / 36, 64 slots 48 / 64 / 169 against 42 / 57 / 124.
  const int32_t pairs = (a.r.group + kVerifyHeads - 1) / kVerifyHeads;
  const int32_t heads = static_cast<int64_t>(m) * a.r.hk * pairs >= 256 ? kVerifyHeads : 1;
  const int32_t chunks = heads == 1 ? a.r.group : pairs;  // workgroups of a k-head
  const dim3 grid(static_cast<unsigned>(a.r.hk * chunks), static_cast<unsigned>(m));
  constexpr int threads = D * 4 * verify_par(NB, D);
  if (a.mma == kPolFP32)  // (one kernel for either activation: fp32 MFMA leaves the vector units idle enough)
    tree_verify_kernel<FullMma, T, K, D, NB, -1><<<grid, threads, 0, s>>>(a, heads, chunks);
  else if (a.silu)
    tree_verify_kernel<PairMma, T, K, D, NB, 1><<<grid, threads, 0, s>>>(a, heads, chunks);
  else
    tree_verify_kernel<PairMma, T, K, D, NB, 0><<<grid, threads, 0, s>>>(a, heads, chunks);
  return hipGetLastError();
}

template <typename T, int K, int D>
hipError_t verify_d(const TreeArgs& a, int32_t m, hipStream_t s) {
  if (a.max_nodes <= 16) return verify_nb<T, K, D, 1>(a, m, s);
  if (a.max_nodes <= 32) return verify_nb<T, K, D, 2>(a, m, s);
  return verify_nb<T, K, D, 4>(a, m, s);
}

template <typename T, int K>
hipError_t verify_k(const TreeArgs& a, int32_t m, hipStream_t s) {
  switch (a.r.d) {
    case 32: return verify_d<T, K, 32>(a, m, s);
    case 64: return verify_d<T, K, 64>(a, m, s);
    default: return verify_d<T, K, 128>(a, m, s);
  }
}

template <typename T>
hipError_t verify_t(const TreeArgs& a, int32_t m, hipStream_t s) {
  switch (a.width) {
    case 2: return verify_k<T, 2>(a, m, s);
    case 3: return verify_k<T, 3>(a, m, s);
    default: return verify_k<T, 4>(a, m, s);
  }
}

// ------------------------------------------------------------------------------- accept

// Bound by HBM: every moved slot's state is read and written once (64 slots of a 16/32-head, d = 128 layer
// in 48.5 us: 250 MB by the counters, 5.2 TB/s; the path's k and u are a few rows from L2). The state rows are
// the first loads, and wait for nothing but the slot's address and number of nodes.
//
// One workgroup per (slot, v-head): wave w takes D / NW state rows, lanes as in the decode kernel (D / 16
// lanes a row, 16 columns each), all of them loaded first; then one rank-one update per path node. The
// workgroups past the heads move the conv state, 8 channels a thread.
template <int D>
struct AcceptCfg {
  static constexpr int LPR = D / 16;
  static constexpr int RPP = kWave / LPR;
  static constexpr int NW = D / RPP < 4 ? D / RPP : 4;
  static constexpr int P = D / (RPP * NW);
};

template <typename T, int K, int D>
__global__ __launch_bounds__(AcceptCfg<D>::NW* kWave) void tree_accept_kernel(AcceptArgs a) {
  using Cfg = AcceptCfg<D>;
  constexpr int LPR = Cfg::LPR, RPP = Cfg::RPP, P = Cfg::P;
  const int i = blockIdx.y;
  int first, n;
  tree_span(a.cu_nodes, i, a.total_nodes, a.max_nodes, first, n);
  const uint64_t sp = ((cu64*)a.state_ptrs)[i];
  const uint64_t cp = ((cu64*)a.conv_ptrs)[i];
  const int last = ((ci32*)a.accepted)[i];
  if (sp == 0 || cp == 0 || last < 0 || last >= n) return;
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= a.hv) {
    // conv state: rows [.. K-3] of the new one are the rows before the node, row K-2 is the node's x
    const int ch0 = ((blockIdx.x - a.hv) * blockDim.x + tid) * 8;
    if (ch0 >= a.channels) return;
    T* cs = reinterpret_cast<T*>(cp) + ch0;
    const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(first) * a.x_stride + ch0;
    typename Vec8<T>::Raw rows[K - 1];  // newest first
    int at = last, row = K - 2;
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      rows[t] = Vec8<T>::load_raw(at >= 0 ? x + at * a.x_stride : cs + static_cast<int64_t>(row) * a.channels);
      if (at >= 0) at = parent_of(a.parents, first, at);
      else --row;
    }
#pragma unroll
    for (int t = 0; t < K - 1; ++t)
      *reinterpret_cast<typename Vec8<T>::Raw*>(cs + static_cast<int64_t>(K - 2 - t) * a.channels) = rows[t];
    return;
  }
  const int lane = tid & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % LPR, rl = lane / LPR;
  const int j = blockIdx.x;
  const int h = j / (a.hv / a.hk);
  const int row0 = w * RPP * P + rl;
  gf32x4* S = (gf32x4*)(reinterpret_cast<float*>(sp) + static_cast<int64_t>(j) * D * D);
  f32x4 s[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s[p][e] = __builtin_nontemporal_load(S + static_cast<int64_t>(row0 + p * RPP) * (D / 4) + c + LPR * e);

  // lane t < n: G_t, and its root path's nodes by doubling the ancestors
  const float gam = lane < n ? a.gamma_rec[static_cast<int64_t>(first + lane) * a.hv + j] : 0.f;
  int up = lane < n ? parent_of(a.parents, first, lane) : -1;
  // sums that started again on the way (restarted_sum): g of every node out of them, summed in two halves
  const bool again = __any(gam < kForget);
  Gamma sum = {gam, 0.f};
  if (again) {
    const float before = __shfl(gam, up >= 0 ? up : 0);
    // (two sums of -inf: finite g whose sum is not)
    sum = gamma_of(up < 0 || (before < kForget && gam > before) ? gam : gam == -__builtin_inff() ? gam : gam - before);
  }
  uint32_t lo = lane < 32 ? 1u << lane : 0u, hi = lane >= 32 ? 1u << (lane - 32) : 0u;
  while (__any(up >= 0)) {
    const int from = up >= 0 ? up : lane;
    const uint32_t lo2 = __shfl(lo, from), hi2 = __shfl(hi, from);
    const int up2 = __shfl(up, from);
    const Gamma s2 = {__shfl(sum.hi, from), __shfl(sum.lo, from)};
    if (up >= 0) {
      lo |= lo2;
      hi |= hi2;
      up = up2;
      if (again) sum = sum + s2;
    }
  }
  uint64_t path = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lo), last)) |
                  static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(hi), last))) << 32;
  // lane t: e^(G_a - G_t), the factor of node t's update
  const float end_hi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum.hi), last));
  const float end_lo = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum.lo), last));
  const float alpha = expf(end_hi) * (1.0f + end_lo);
  const float f = expf((end_hi - sum.hi) + (end_lo - sum.lo));
  const f32x4* kb = reinterpret_cast<const f32x4*>(a.k_rec + (static_cast<int64_t>(first) * a.hk + h) * D) + c;
  const float* ub = a.u_rec + (static_cast<int64_t>(first) * a.hv + j) * D + row0;
  const int64_t kstep = static_cast<int64_t>(a.hk) * (D / 4), ustep = static_cast<int64_t>(a.hv) * D;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[p][e][q] *= alpha;
  // the path in order, BATCH nodes' k and u loaded before the first is used (past the path's end the last
  // one's again, unused)
  constexpr int BATCH = 4;
  while (path) {
    f32x4 kv[BATCH][4];
    float uv[BATCH][P], fv[BATCH];
    bool have[BATCH];
    int t = 0;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      have[b] = path != 0;
      t = have[b] ? __builtin_ctzll(path) : t;
      path &= path - 1;
      fv[b] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), t));
#pragma unroll
      for (int e = 0; e < 4; ++e) kv[b][e] = kb[t * kstep + LPR * e];
#pragma unroll
      for (int p = 0; p < P; ++p) uv[b][p] = ub[t * ustep + p * RPP];
    }
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
      if (!have[b]) break;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float u = fv[b] * uv[b][p];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int q = 0; q < 4; ++q) s[p][e][q] = fmaf(u, kv[b][e][q], s[p][e][q]);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_nontemporal_store(s[p][e], S + static_cast<int64_t>(row0 + p * RPP) * (D / 4) + c + LPR * e);
}

template <typename T, int K, int D>
hipError_t accept_d(const AcceptArgs& a, int32_t m, hipStream_t s) {
  constexpr int threads = AcceptCfg<D>::NW * kWave;
  const int conv_blocks = (a.channels / 8 + threads - 1) / threads;
  const dim3 grid(static_cast<unsigned>(a.hv + conv_blocks), static_cast<unsigned>(m));
  tree_accept_kernel<T, K, D><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int K>
hipError_t accept_k(const AcceptArgs& a, int32_t m, hipStream_t s) {
  switch (a.d) {
    case 32: return accept_d<T, K, 32>(a, m, s);
    case 64: return accept_d<T, K, 64>(a, m, s);
    default: return accept_d<T, K, 128>(a, m, s);
  }
}

template <typename T>
hipError_t accept_t(const AcceptArgs& a, int32_t m, hipStream_t s) {
  switch (a.width) {
    case 2: return accept_k<T, 2>(a, m, s);
    case 3: return accept_k<T, 3>(a, m, s);
    default: return accept_k<T, 4>(a, m, s);
  }
}

}  // namespace

hipError_t launch_tree_verify(const TreeArgs& a, int32_t m, hipStream_t s) {
  if (m == 0) return hipSuccess;
  return a.bf16 ? verify_t<uint16_t>(a, m, s) : verify_t<float>(a, m, s);
}

hipError_t launch_tree_accept(const AcceptArgs& a, int32_t m, hipStream_t s) {
  if (m == 0) return hipSuccess;
  return a.bf16 ? accept_t<uint16_t>(a, m, s) : accept_t<float>(a, m, s);
}

}  // namespace gdn
