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

// Slot i's rows: the first, and how many the call works on (none where cu_nodes does not lie
// inside [0, total]).
__device__ __forceinline__ void tree_span(const int32_t* cu, int i, int total, int max_nodes, int& first, int& n) {
  const int b = ((ci32*)cu)[i], e = ((ci32*)cu)[i + 1];
  first = b;
  n = 0;
  if (b < 0 || e <= b || b >= total) return;
  n = e - b < max_nodes ? e - b : max_nodes;
  n = n < total - b ? n : total - b;
}

// Node t's parent inside its tree (-1: the slot itself).
__device__ __forceinline__ int parent_of(const int32_t* parents, int first, int t) {
  if (t < 0) return -1;
  if (!parents) return t - 1;
  const int p = parents[first + t];
  return p >= -1 && p < t ? p : -1;
}

// Renumbers grid.x so that consecutive v-heads, which read the same q and k channels, share an
// XCD's L2 (see decode.hip).
__device__ __forceinline__ int xcd_head() {
  const int n = gridDim.x, b = blockIdx.x;
  return (n % 8 == 0) ? (b % 8) * (n / 8) + b / 8 : b;
}

// One workgroup per (slot, v-head), one wave per 16 state rows; NB = blocks of 16 nodes.
//
// The rows of the state do not mix, so with K, Q [N][d] the normalised tokens and S the wave's 16
// rows everything is small matrix products, on 16x16 fp32 MFMA tiles whose contraction index runs
// as 4 (l / 16) + r: the tile of a result (lane l: rows 4 (l / 16) + r of column l % 16) is then the
// right operand of the next product as it stands.
//   M = K S^T, W = Q S^T               [N][16]
//   A_ij = -beta_i e^(G_i - G_j) k_i.k_j for j above i, else 0;   P_ij = e^(G_i - G_j) q_i.k_j, j above or at i
//   U = (I - A)^-1 (beta (V - e^G M)), O = e^G W + P U
// (I - A) is unit lower triangular (parents come first): its 16x16 diagonal blocks are inverted by
// substitution, the rest is block substitution on MFMA.
//
// A zero of A or P times an infinity or a NaN would carry a broken token into branches that do not
// see it. So such values never enter the products: a k that is not finite marks its node, a right
// side beta (v - e^G M) that is not finite marks its node for that state row, zeros go in their
// place, and the results of the marked nodes and their descendants are set to NaN at the end.
template <typename T, int K, int D, int NB, bool SILU>
__global__ __launch_bounds__(D * 4) void tree_verify_kernel(TreeArgs a) {
  constexpr int W = D / 16;          // waves
  constexpr int NT = W * kWave;      // threads (4 D)
  constexpr int N = 16 * NB;
  constexpr int KS = D + 4;          // floats of an LDS row of K and Q
  constexpr int PS = N + 4;          // floats of an LDS row of A and P
  constexpr int CH = 2 * D / 8;      // 8-channel pieces of a node's k-head channels (q, then k)
  __shared__ __attribute__((aligned(16))) float qk_l[2][N][KS];  // q^, k^
  __shared__ __attribute__((aligned(16))) float a_l[N][PS];      // A
  __shared__ __attribute__((aligned(16))) float p_l[N][PS];      // P
  __shared__ __attribute__((aligned(16))) float t_l[NB][16][20]; // inverses of the diagonal blocks
  __shared__ float gam_l[N], eg_l[N], beta_l[N];
  __shared__ uint32_t anc_l[N][2];                               // ancestors (bit j: node j), not itself
  __shared__ uint32_t kbad_l[2], qbad_l[2];                      // nodes whose k (q) is not finite
  __shared__ int par_l[N];
  __shared__ int win_l[N][3];  // the rows before node i, newest first: a node, or -1 - r for conv-state row r

  const RecurArgs& r = a.r;
  const int i = blockIdx.y;
  const int j = xcd_head();
  int first, n;
  tree_span(a.cu_nodes, i, a.total_nodes, a.max_nodes, first, n);
  const uint64_t sp = ((cu64*)r.state_ptrs)[i];
  const uint64_t cp = ((cu64*)a.conv_ptrs)[i];
  if (n == 0 || sp == 0 || cp == 0) return;  // (the whole workgroup)
  const int tid = threadIdx.x;
  const int lane = tid & (kWave - 1);
  const int w = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c4 = lane / 16, l16 = lane % 16;
  const int h = j / r.group;
  const int C = a.channels;

  // the wave's state rows: lane (c4, l16) holds columns 16 e + 4 c4 .. + 3 of row l16
  const gf32x4* S = (const gf32x4*)(reinterpret_cast<const float*>(sp) +
                                    (static_cast<int64_t>(j) * D + w * 16 + l16) * D);
  f32x4 s[D / 16];
#pragma unroll
  for (int e = 0; e < D / 16; ++e) s[e] = __builtin_nontemporal_load(S + 4 * e + c4);

  if (tid < N) {
    const bool live = tid < n;
    par_l[tid] = live ? parent_of(a.parents, first, tid) : -1;
    const int64_t gi = static_cast<int64_t>(first + tid) * r.hv + j;
    gam_l[tid] = live ? r.g[gi] : 0.f;
    beta_l[tid] = live ? r.beta[gi] : 0.f;
  }
  if (tid < 2) kbad_l[tid] = qbad_l[tid] = 0;
  __syncthreads();
  if (tid < N) {
    // walk K-1 rows back: nodes up to the root, then conv-state rows, newest (K-2) first
    int at = par_l[tid], row = K - 2;
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
      win_l[tid][t] = at >= 0 ? at : -1 - row;
      if (at >= 0) at = par_l[at];
      else --row;
    }
  }
  if (w == 0) {
    // ancestors and sums of g along the root path by doubling: after round s they cover 2^s levels
    const bool live = lane < N;
    int up = live ? par_l[lane] : -1;
    float gam = live ? gam_l[lane] : 0.f;
    uint32_t lo = up >= 0 && up < 32 ? 1u << up : 0u, hi = up >= 32 ? 1u << (up - 32) : 0u;
#pragma unroll
    for (int s2 = 1; s2 < N; s2 *= 2) {
      const int from = up >= 0 ? up : lane;
      const uint32_t lo2 = __shfl(lo, from), hi2 = __shfl(hi, from);
      const float g2 = __shfl(gam, from);
      const int up2 = __shfl(up, from);
      if (up >= 0) {
        lo |= lo2;
        hi |= hi2;
        gam += g2;
        up = up2;
      }
    }
    if (live) {
      anc_l[lane][0] = lo;
      anc_l[lane][1] = hi;
      gam_l[lane] = gam;
      eg_l[lane] = expf(gam);
      if (lane < n && a.gamma_rec) a.gamma_rec[static_cast<int64_t>(first + lane) * r.hv + j] = gam;
    }
  }
  __syncthreads();

  const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(first) * a.x_stride;
  const T* cs = reinterpret_cast<const T*>(cp);
  // q and k of every node: a thread convolves 8 channels (always the same ones) of one node a
  // pass, 2 D / 8 threads a node
  {
    const int piece = tid % CH;
    const bool is_k = piece * 8 >= D;
    const int d0 = (piece * 8) % D;
    const int ch0 = (is_k ? r.hk * D : 0) + h * D + d0;
    ConvTaps<T, K> taps;
    taps.load(static_cast<const T*>(a.w), static_cast<const T*>(a.b), ch0);
#pragma unroll
    for (int pass = 0; pass < N / (NT / CH); ++pass) {
      const int t = pass * (NT / CH) + tid / CH;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < n) {
        float win[K - 1][8], cur[8];
#pragma unroll
        for (int q = 0; q < K - 1; ++q) {
          const int at = win_l[t][K - 2 - q];
          Vec8<T>::load(at >= 0 ? x + at * a.x_stride + ch0 : cs + static_cast<int64_t>(-1 - at) * C + ch0, win[q]);
        }
        Vec8<T>::load(x + t * a.x_stride + ch0, cur);
        taps.apply(win, cur, SILU, y);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      ss = group_sum<D / 8>(ss);
      float f = r.qk_norm && t < n ? 1.0f / sqrtf(ss + r.eps) : 1.0f;
      if (!is_k) f *= r.scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= f;
      if (t < n && is_k && a.k_rec && j % r.group == 0)
        Vec8<float>::store(a.k_rec + (static_cast<int64_t>(first + t) * r.hk + h) * D + d0, y);
      if (!(ss < __builtin_inff())) {  // (the node's threads agree on ss)
        float bad = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) bad += y[e] * 0.f;
        if (group_sum<D / 8>(bad) != 0.f) {
          atomicOr(&(is_k ? kbad_l : qbad_l)[t >> 5], 1u << (t & 31));
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = 0.f;
        }
      }
      float* dst = &qk_l[is_k ? 1 : 0][t][d0];
      *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
  // v of the lane's nodes (4 c4 + 0..3 of every block) at its state row
  float v[NB][4];
  {
    const int ch = (2 * r.hk + j) * D + w * 16 + l16;
    float tap[K];
#pragma unroll
    for (int t = 0; t < K; ++t) tap[t] = elem_f32<T>(static_cast<const T*>(a.w)[static_cast<int64_t>(ch) * K + t]);
    const float bias = a.b ? elem_f32<T>(static_cast<const T*>(a.b)[ch]) : 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 16 * b + 4 * c4 + e;
        v[b][e] = 0.f;
        if (t < n) {
          float acc = bias;
#pragma unroll
          for (int q = 0; q < K - 1; ++q) {
            const int at = win_l[t][K - 2 - q];
            acc = fmaf(tap[q], elem_f32<T>(at >= 0 ? x[at * a.x_stride + ch] : cs[static_cast<int64_t>(-1 - at) * C + ch]),
                       acc);
          }
          acc = fmaf(tap[K - 1], elem_f32<T>(x[t * a.x_stride + ch]), acc);
          v[b][e] = SILU ? silu(acc) : acc;
        }
      }
  }
  __syncthreads();

  // A and P: the lower blocks of k k^T and q k^T, dealt to the waves
  {
    constexpr int NL = NB * (NB + 1) / 2;
    for (int task = w; task < 2 * NL; task += W) {
      const bool is_p = task >= NL;
      int bi = 0, rest = is_p ? task - NL : task;
      while (rest > bi) rest -= ++bi;  // block row bi, block column rest
      const int bj = rest;
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const f32x4 left = *reinterpret_cast<const f32x4*>(&qk_l[is_p ? 0 : 1][16 * bi + l16][16 * e + 4 * c4]);
        const f32x4 right = *reinterpret_cast<const f32x4*>(&qk_l[1][16 * bj + l16][16 * e + 4 * c4]);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(left[q], right[q], acc, 0, 0, 0);
      }
      const int col = 16 * bj + l16;
      const float gcol = gam_l[col];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 16 * bi + 4 * c4 + q;
        const bool above = (anc_l[row][col >> 5] >> (col & 31)) & 1u;
        const bool use = above || (is_p && row == col);
        const float f = use ? expf(gam_l[row] - gcol) * (is_p ? 1.0f : -beta_l[row]) : 0.f;
        (is_p ? p_l : a_l)[row][col] = use ? f * acc[q] : 0.f;
      }
    }
  }
  __syncthreads();
  // inverses of the diagonal blocks: lane 16 b + c of the first wave forms column c of block b
  if (w == 0 && lane < N) {
    const int b = lane / 16;
    float col[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      float acc = q == l16 ? 1.0f : 0.0f;
#pragma unroll
      for (int t = 0; t < q; ++t) acc = fmaf(a_l[16 * b + q][16 * b + t], col[t], acc);
      col[q] = acc;
      t_l[b][q][l16] = acc;
    }
  }
  // M and W
  f32x4 m[NB], o[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) m[b] = o[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const f32x4 qf = *reinterpret_cast<const f32x4*>(&qk_l[0][16 * b + l16][16 * e + 4 * c4]);
      const f32x4 kf = *reinterpret_cast<const f32x4*>(&qk_l[1][16 * b + l16][16 * e + 4 * c4]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        m[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(kf[q], s[e][q], m[b], 0, 0, 0);
        o[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(qf[q], s[e][q], o[b], 0, 0, 0);
      }
    }
  __syncthreads();
  // block substitution; u of block b replaces m[b]
  const int64_t base = (static_cast<int64_t>(first) * r.hv + j) * D + w * 16 + l16;
  uint32_t bad[2] = {kbad_l[0], kbad_l[1]};  // marked nodes of the lane's state row
  const uint32_t qbad[2] = {qbad_l[0], qbad_l[1]};
  bool dirty = (bad[0] | bad[1] | qbad[0] | qbad[1]) != 0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    f32x4 rhs, eg;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * b + 4 * c4 + q;
      eg[q] = eg_l[t];
      rhs[q] = beta_l[t] * (v[b][q] - eg[q] * m[b][q]);
      o[b][q] *= eg[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t off = __ballot(!(fabsf(rhs[q]) < __builtin_inff()));
      if (off) {
        dirty = true;
#pragma unroll
        for (int g = 0; g < 4; ++g)
          if ((off >> (16 * g + l16)) & 1u) bad[b / 2] |= 1u << (16 * (b % 2) + 4 * g + q);
        if ((off >> lane) & 1u) rhs[q] = 0.f;
      }
    }
#pragma unroll
    for (int b2 = 0; b2 < b; ++b2) {
      const f32x4 left = *reinterpret_cast<const f32x4*>(&a_l[16 * b + l16][16 * b2 + 4 * c4]);
#pragma unroll
      for (int q = 0; q < 4; ++q) rhs = __builtin_amdgcn_mfma_f32_16x16x4f32(left[q], m[b2][q], rhs, 0, 0, 0);
    }
    const f32x4 inv = *reinterpret_cast<const f32x4*>(&t_l[b][l16][4 * c4]);
    f32x4 u = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 4; ++q) u = __builtin_amdgcn_mfma_f32_16x16x4f32(inv[q], rhs[q], u, 0, 0, 0);
    m[b] = u;
#pragma unroll
    for (int b2 = 0; b2 <= b; ++b2) {
      const f32x4 left = *reinterpret_cast<const f32x4*>(&p_l[16 * b + l16][16 * b2 + 4 * c4]);
#pragma unroll
      for (int q = 0; q < 4; ++q) o[b] = __builtin_amdgcn_mfma_f32_16x16x4f32(left[q], m[b2][q], o[b], 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = 16 * b + 4 * c4 + q;
      if (dirty) {
        const uint32_t self = 1u << (t & 31);
        const bool hit = (((anc_l[t][0] | (t < 32 ? self : 0u)) & bad[0]) | ((anc_l[t][1] | (t < 32 ? 0u : self)) & bad[1])) != 0;
        if (hit) u[q] = __builtin_nanf("");
        if (hit || (qbad[t >> 5] & self)) o[b][q] = __builtin_nanf("");
      }
      if (t < n) {
        const int64_t at = base + static_cast<int64_t>(t) * r.hv * D;
        if (r.o_bf16)
          static_cast<uint16_t*>(r.o)[at] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[b][q]));
        else
          static_cast<float*>(r.o)[at] = o[b][q];
        if (a.u_rec) a.u_rec[at] = u[q];
      }
    }
  }
}

template <typename T, int K, int D, int NB>
hipError_t verify_nb(const TreeArgs& a, int32_t m, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.r.hv), static_cast<unsigned>(m));
  if (a.silu)
    tree_verify_kernel<T, K, D, NB, true><<<grid, D * 4, 0, s>>>(a);
  else
    tree_verify_kernel<T, K, D, NB, false><<<grid, D * 4, 0, s>>>(a);
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

  // lane t < n: is node t on the path? bits of the path by doubling the ancestors
  int up = lane < n ? parent_of(a.parents, first, lane) : -1;
  uint32_t lo = lane < 32 ? 1u << lane : 0u, hi = lane >= 32 ? 1u << (lane - 32) : 0u;
  for (int s2 = 1; s2 < n; s2 *= 2) {
    const int from = up >= 0 ? up : lane;
    const uint32_t lo2 = __shfl(lo, from), hi2 = __shfl(hi, from);
    const int up2 = __shfl(up, from);
    if (up >= 0) {
      lo |= lo2;
      hi |= hi2;
      up = up2;
    }
  }
  uint64_t path = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(lo), last)) |
                  static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(hi), last))) << 32;
  const float* gam = a.gamma_rec + static_cast<int64_t>(first) * a.hv + j;
  const float gend = gam[static_cast<int64_t>(last) * a.hv];
  const float alpha = expf(gend);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[p][e][q] *= alpha;
  while (path) {
    const int t = __builtin_ctzll(path);
    path &= path - 1;
    const int64_t node = first + t;
    const float f = expf(gend - gam[static_cast<int64_t>(t) * a.hv]);
    const f32x4* kp = reinterpret_cast<const f32x4*>(a.k_rec + (node * a.hk + h) * D);
    const float* up_ = a.u_rec + (node * a.hv + j) * D + row0;
    f32x4 kv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) kv[e] = kp[c + LPR * e];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float u = f * up_[p * RPP];
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[p][e][q] = fmaf(u, kv[e][q], s[p][e][q]);
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
