// Trees of drafted tokens over the recurrent state, and the commit of an
// accepted path, on gfx950.
//
// A node's output is the recurrence's output after the tokens on its path, so
// with S the state, E_i the product of the decays on node i's path (per key
// channel) and anc(i) its ancestors, unrolling S_t = Diag(a) S + k d^T along
// the path gives
//   d_i = beta_i (v_i - S^T (E_i k_i) - sum_{j in anc(i)} A_ij d_j),
//         A_ij = sum_c k_ic (E_ic / E_jc) k_jc
//   o_i = scale (S^T (E_i q_i) + sum_{j in anc(i)} B_ij d_j + (q_i . k_i) d_i),
//         B_ij = sum_c q_ic (E_ic / E_jc) k_jc
// No node's state is ever formed: S is read once and only the rows d_i (one
// vector of D values per node) take the states' place.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

constexpr int kMaxNodes = KDA_TREE_MAX_NODES;

// Lane rotations and broadcasts inside rows of 16 lanes, as operand modifiers
// of vector instructions (no LDS crossbar, which all waves of a CU share).
template <int kCtrl>
__device__ __forceinline__ float row_dpp(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), kCtrl, 0xF, 0xF, true));
}
template <int R> __device__ __forceinline__ float row_ror(float x) { return row_dpp<0x120 + R>(x); }
template <int L> __device__ __forceinline__ float row_bcast(float x) { return row_dpp<0x150 + L>(x); }

// Sum over the 64 lanes, as a wave-uniform value.
__device__ __forceinline__ float wave_sum(float x) {
  x += row_ror<8>(x); x += row_ror<4>(x); x += row_ror<2>(x); x += row_ror<1>(x);
  // rows 1 and 3 take rows 0 and 2 in, then rows 2 and 3 row 1's sum
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x142, 0xA, 0xF, false));
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x143, 0xC, 0xF, false));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Two consecutive elements in one load (p even-aligned), as floats when needed.
template <typename T> struct Pair;
template <> struct Pair<bf16_bits> {
  uint32_t w;
  __device__ __forceinline__ void load(const bf16_bits* p) { w = *(const uint32_t*)p; }
  __device__ __forceinline__ float get(int c) const {
    return __builtin_bit_cast(float, c ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ void store(bf16_bits* p, float a, float b) {
    const bf16x4 y = to_bf16x4(f32x4{a, b, 0.f, 0.f});
    *(uint32_t*)p = __builtin_bit_cast(uint2, y).x;
  }
};
template <> struct Pair<float> {
  f32x2 w;
  __device__ __forceinline__ void load(const float* p) { w = *(const f32x2*)p; }
  __device__ __forceinline__ float get(int c) const { return w[c]; }
  static __device__ __forceinline__ void store(float* p, float a, float b) { *(f32x2*)p = f32x2{a, b}; }
};

// kN consecutive elements (a multiple of 16 bytes) in 16-byte loads.
template <typename T, int kN> struct Run {
  u32x4 w[kN * sizeof(T) / 16];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (int)(kN * sizeof(T) / 16); ++i) w[i] = ((const u32x4*)p)[i];
  }
  __device__ __forceinline__ float get(int c) const {
    if constexpr (sizeof(T) == 4) {
      return __builtin_bit_cast(float, (uint32_t)w[c / 4][c % 4]);
    } else {
      const uint32_t d = w[c / 8][c / 2 % 4];
      return __builtin_bit_cast(float, c % 2 ? d & 0xffff0000u : d << 16);
    }
  }
};

// One element, with the interface of Pair.
template <typename T> struct One {
  T w;
  __device__ __forceinline__ void load(const T* p) { w = *p; }
  __device__ __forceinline__ float get(int) const { return Elem<T>::load(&w); }
  static __device__ __forceinline__ void store(T* p, float a, float) { Elem<T>::store(p, a); }
};

// Decay of one channel of token row `row` (a row of the [N, T, H] grid). The
// clamps of gate_alpha drop a NaN, which is kept here.
__device__ __forceinline__ float load_alpha(const float* g, int gate, size_t row, int D, int c, uint32_t fe_flags,
                                            float g_min, float alpha_min) {
  if (gate == KDA_GATE_NONE) return 1.f;
  const float x = g[gate == KDA_GATE_CHANNEL ? row * D + c : row];
  if (x != x) return x;
  return fe_flags & KDA_FE_GATE_LOGITS ? gate_alpha_logit(x, alpha_min) : gate_alpha(x, g_min);
}

// The parent of node i as the kernels use it: -1 unless in [0, i - 1].
__device__ __forceinline__ int clean_parent(const int32_t* parents, size_t first, int i) {
  if (!parents) return i - 1;
  const int p = parents[first + i];
  return p >= 0 && p < i ? p : -1;
}

// The tree of one sequence as a wave holds it (lane i is node i): every node's
// ancestors and itself as a bit mask, by doubling the distance looked back.
__device__ __forceinline__ uint64_t ancestors(int parent, int lane) {
  uint64_t anc = 1ull << lane;
  for (int jump = parent; __ballot(jump >= 0);) {
    const uint64_t up = __shfl((unsigned long long)anc, max(jump, 0));
    const int next = __shfl(jump, max(jump, 0));
    if (jump >= 0) { anc |= up; jump = next; }
  }
  return anc;
}

// Decays between nodes as quotients E_i / E_j of the decays from the state.
// Where every E of any tree of T nodes is at least 2^-kMaxSpan, far inside the
// range of fp32, they are formed as they stand.
// Otherwise G = log2 E is kept in fp64 and referred, per block of 16 rows and
// channel, to R half way between the block's largest and smallest G:
//   E_i / E_j = 2^(G_i - R) 2^(R - G_j).
// The first exponent is at most half the block's spread in size, and so is the
// second from above whenever j is an ancestor of a node of the block (from
// below it may underflow, as the quotient does). So only the spread inside a
// block is limited, not the depth of the tree. What exceeds that too (a floor
// below -5.2 with chains of 16, blocks that mix deep and shallow branches) is
// left to the path kernel; both kernels decide it from the tree alone.
constexpr float kMaxSpan = 87.f;      // log2 (2^-87 = e^-60)
constexpr float kMaxSpread = 120.f;   // log2: factors reach 2^60

// 2^x, x any finite fp64: the integer part goes to the exponent, so that a
// large x costs no digits. Overflows to infinity, underflows to 0.
__device__ __forceinline__ float exp2_wide(double x) {
  const double i = rint(fmin(fmax(x, -400.0), 400.0));
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(fmin(fmax(x, -400.0), 400.0) - i)), (int)i);
}

// log2 of the decay of one channel.
__device__ __forceinline__ double log2_alpha(float g, bool logits, float g_min) {
  const double l2e = 1.4426950408889634074;
  if (!logits) return (double)fminf(fmaxf(g, g_min), 0.f) * l2e;
  // -softplus(a) = min(-a, 0) - ln(1 + e^-|a|)
  const float soft = fminf(-g, 0.f) - log1pf(__builtin_amdgcn_exp2f(-fabsf(g) * kLog2e));
  return (double)fmaxf(soft, g_min) * l2e;
}

// Largest depth of a block's nodes below their deepest common ancestor, over
// the blocks: the number of decays a block's spread consists of, at most.
__device__ __forceinline__ int block_depth(uint64_t anc, bool live) {
  uint64_t common = live ? anc : ~0ull;
  int deep = live ? __builtin_popcountll(anc) : 0;
#pragma unroll
  for (int m = 1; m < 16; m *= 2) {
    common &= __shfl_xor((unsigned long long)common, m);
    deep = max(deep, __shfl_xor(deep, m));
  }
  int most = deep ? deep - __builtin_popcountll(common) : 0;
  most = max(most, __shfl_xor(most, 16));
  return max(most, __shfl_xor(most, 32));
}
// How many decays at the floor stay within `span` (log2), at most kMaxNodes.
static int reach_of(float span, float g_min, int gate) {
  if (gate == KDA_GATE_NONE || g_min == 0.f) return kMaxNodes;
  const float r = span / (-g_min * kLog2e);
  return r >= (float)kMaxNodes ? kMaxNodes : (int)r;
}

constexpr int kNoneTaken = -1;

// ---- any decays, any head size -------------------------------------------------
// One 256-thread workgroup per (sequence, head). A_ij and B_ij are summed pair
// by pair along each node's path, with the decay between the two nodes built
// up factor by factor on the way to the root, so no quotient of decays is ever
// formed and any floor works; only a node's own ancestors are touched. Bound by
// its sums over the lanes, two for each (node, ancestor) pair: for the trees
// that the other kernels cannot take.
// LDS, fp32: k, q, alpha [T][D], A, B [T][T].
template <int D>
constexpr size_t path_lds_bytes(int T) {
  return sizeof(float) * ((size_t)3 * T * D + 2 * T * T + 2 * kMaxNodes);
}

template <int D, typename TIn>
__global__ __launch_bounds__(256) void tree_path_kernel(
    const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
    const float* __restrict__ g, const float* __restrict__ beta, const float* __restrict__ state,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes, TIn* __restrict__ o, int H,
    int T, float scale, float g_min, uint32_t fe_flags, float fe_eps, int gate, int taken) {
  const uint32_t n = blockIdx.x / (uint32_t)H, h = blockIdx.x % (uint32_t)H;
  const int nt = num_nodes ? min(max(num_nodes[n], 0), T) : T;
  if (nt == 0) return;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
  if (taken != kNoneTaken) {   // sequences whose blocks are no deeper are another kernel's
    const int p = lane < nt ? clean_parent(parents, (size_t)n * T, lane) : -1;
    if (block_depth(ancestors(p, lane), lane < nt) <= taken) return;
  }
  extern __shared__ float smem[];
  float* s_k = smem;
  float* s_q = s_k + T * D;
  float* s_a = s_q + T * D;                 // alpha, then E, then d
  float* s_A = s_a + T * D;
  float* s_B = s_A + T * T;
  int* s_par = (int*)(s_B + T * T);
  float* s_b = (float*)(s_par + kMaxNodes);
  auto row = [&](int t) __attribute__((always_inline)) { return ((size_t)n * T + t) * H + h; };

  const float alpha_min = __builtin_amdgcn_exp2f(g_min * kLog2e);
  const bool norm = fe_flags & KDA_FE_L2NORM_QK;
  if (tid < nt) {
    s_par[tid] = clean_parent(parents, (size_t)n * T, tid);
    const float b = beta[row(tid)];
    s_b[tid] = fe_flags & KDA_FE_BETA_LOGITS ? beta_logit(b) : b;
  }
  // one wave per node: lane l stages channels l and l + 64
  for (int i = wave; i < nt; i += 4) {
    float kv[2] = {0.f, 0.f}, qv[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = lane + 64 * x;
      if (c < D) {
        kv[x] = Elem<TIn>::load(k + row(i) * D + c);
        qv[x] = Elem<TIn>::load(q + row(i) * D + c);
        s_a[i * D + c] = load_alpha(g, gate, row(i), D, c, fe_flags, g_min, alpha_min);
      }
    }
    if (norm) {
      const float rk = inv_norm(wave_sum(kv[0] * kv[0] + kv[1] * kv[1]), fe_eps);
      const float rq = inv_norm(wave_sum(qv[0] * qv[0] + qv[1] * qv[1]), fe_eps);
      kv[0] *= rk; kv[1] *= rk; qv[0] *= rq; qv[1] *= rq;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = lane + 64 * x;
      if (c < D) { s_k[i * D + c] = kv[x]; s_q[i * D + c] = qv[x]; }
    }
  }
  __syncthreads();

  // A and B, one wave per node, walking to the root; r: decay from j to i
  for (int i = wave; i < nt; i += 4) {
    float ki[2] = {0.f, 0.f}, qi[2] = {0.f, 0.f}, r[2] = {0.f, 0.f};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int c = lane + 64 * x;
      if (c < D) { ki[x] = s_k[i * D + c]; qi[x] = s_q[i * D + c]; r[x] = s_a[i * D + c]; }
    }
    const float self = wave_sum(qi[0] * ki[0] + qi[1] * ki[1]);
    if (lane == 0) s_B[i * T + i] = self;
    for (int j = s_par[i]; j >= 0; j = s_par[j]) {
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = lane + 64 * x;
        if (c < D) {
          const float kj = s_k[j * D + c] * r[x];
          a += ki[x] * kj;
          b += qi[x] * kj;
          r[x] *= s_a[j * D + c];
        }
      }
      a = wave_sum(a);
      b = wave_sum(b);
      if (lane == 0) { s_A[i * T + j] = a; s_B[i * T + j] = b; }
    }
  }
  __syncthreads();

  // E in place of alpha, one thread per channel; then k and q times E
  if (tid < D)
    for (int i = 0; i < nt; ++i) {
      const int p = s_par[i];
      if (p >= 0) s_a[i * D + tid] *= s_a[p * D + tid];
    }
  __syncthreads();
  for (int e = tid; e < nt * D; e += 256) { s_k[e] *= s_a[e]; s_q[e] *= s_a[e]; }

  // Thread (group, column): the state's column in registers
  constexpr int kGroups = 256 / D;
  const int col = tid % D, grp = tid / D;
  const float* S = state + (size_t)blockIdx.x * D * D;
  float s[D];
#pragma unroll
  for (int c = 0; c < D; ++c) s[c] = S[c * D + col];
  __syncthreads();
  float* s_d = s_a;
  // (S^T k)_col of every node, the nodes shared out over the groups
  for (int i = grp; i < nt; i += kGroups) {
    float u = 0.f;
#pragma unroll
    for (int c = 0; c < D; ++c) u += s_k[i * D + c] * s[c];
    s_d[i * D + col] = u;
  }
  __syncthreads();
  if (grp == 0)
    for (int i = 0; i < nt; ++i) {
      float x = Elem<TIn>::load(v + row(i) * D + col) - s_d[i * D + col];
      for (int j = s_par[i]; j >= 0; j = s_par[j]) x -= s_A[i * T + j] * s_d[j * D + col];
      s_d[i * D + col] = s_b[i] * x;
    }
  __syncthreads();
  for (int i = grp; i < nt; i += kGroups) {
    float w = 0.f;
#pragma unroll
    for (int c = 0; c < D; ++c) w += s_q[i * D + c] * s[c];
    for (int j = i; j >= 0; j = s_par[j]) w += s_B[i * T + j] * s_d[j * D + col];
    Elem<TIn>::store(o + row(i) * D + col, scale * w);
  }
}

// ---- D = 128, decays of moderate span ---------------------------------------------
// The same products as tiles of 16 nodes on the matrix cores. One workgroup of
// kWaves waves per (sequence, head); wave w owns the 128 / kWaves value columns
// from there on, and nothing of S, d or o leaves its registers:
//   1. E by products along the paths (doubling), k E, q E and k / E to LDS;
//   2. U = (k E) S and W = (q E) S, S straight from memory in operand layout;
//      A = (k E)(k / E)^T and B = (q E)(k / E)^T, masked to ancestors, to LDS;
//   3. (I + beta A)^-1 of the 16 x 16 diagonal blocks, one row per lane;
//   4. d by blocks of 16 nodes, then o = W + B d. The accumulator layout of a
//      16 x 16 tile is the K = 16 operand layout, so d feeds the products as it is.
// All products use the fp32 matrix instructions, for bf16 tensors too: S, the
// decayed rows, A, B and d have 24 bits whatever the tensors have. Operands of
// two bf16 terms (16 bits, less than a fifth of the matrix time) took 133 to 142
// us for 256 x 32 heads of 16 nodes and 97 to 114 for 64 x 32 heads of 64, but
// rounded 0.5 % of the outputs the other way (now 0.02 %); three terms (24 bits)
// 160 and 180, with the fp32 instructions 167 and 175 on the same card.
// Measured: 256 x 32 heads, 16 nodes, bf16 154 to 187 us (739 MB, 4.0 to 4.8
// TB/s), 128 x 32 heads, 32 nodes 158 to 179 us, 64 x 32 heads, 64 nodes 160 to
// 175 us (336 MB); the products alone would take 70, 77 and 90 us at the rate of
// a large fp32 matrix product (154 TFLOP/s). Bound by loads and products that
// overlap only in part, since a workgroup does first the ones and then the
// others. One sequence of 32 heads and 8 nodes 9 us.
//
// Values that are not finite: a product over nodes would carry one node's NaN
// to nodes that do not descend from it (0 * NaN). So they are replaced by 0
// before such a product and remembered as bits, per node where they reach every
// column (A, B, NaN decays) and per node and column (d); the outputs of their
// nodes and descendants are then set to NaN.

// Operands of products on the fp32 matrix instructions (16 x 16 x 4).
struct FloatOp {
  static constexpr int kRowBytes = 528;               // a row of 128, padded by 16 bytes
  struct F8 { float x[8]; };
  struct F4 { f32x4 x; };
  static __device__ __forceinline__ F8 make8(const float (&x)[8]) {
    F8 f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.x[j] = x[j];
    return f;
  }
  static __device__ __forceinline__ F4 make4(f32x4 x) { return {x}; }
  template <int kN>
  static __device__ __forceinline__ void put(char* row, int c, const float (&x)[kN]) {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i)
      *(f32x4*)(row + 4 * (c + 4 * i)) = f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
  }
  static __device__ __forceinline__ F8 get8(const char* row, int c) {
    F8 f;
    *(f32x4*)f.x = *(const f32x4*)(row + 4 * c);
    *(f32x4*)(f.x + 4) = *(const f32x4*)(row + 4 * c + 16);
    return f;
  }
  static __device__ __forceinline__ void put1(char* m, int stride, int i, int j, float x) {
    ((float*)m)[i * stride + j] = x;
  }
  static __device__ __forceinline__ F4 get4(const char* m, int stride, int i, int j) {
    return {*(const f32x4*)(m + 4 * (i * stride + j))};
  }
  // K is walked in four lane groups an instruction; which of the fragment's
  // elements go together is free as long as both operands agree
  static __device__ __forceinline__ f32x4 mma(const F8& a, const F8& b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[j], b.x[j], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ f32x4 mma(const F4& a, const F4& b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.x[j], b.x[j], c, 0, 0, 0);
    return c;
  }
};

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < __builtin_inff(); }

// kTB: tiles of 16 nodes; kWaves: 4 or 8. With three or four tiles the three
// operand planes would leave room for one workgroup per compute unit, which
// then either loads or computes: q E takes the place of k E once A and U are
// formed, and the matrices lie over the planes (two workgroups; 64 nodes on 64
// x 32 heads: 210 us with one, 173 with two). With one or two tiles all lie side
// by side and two barriers are saved.
template <int kTB, bool kDeep>
struct TileLds {
  using Op = FloatOp;
  static constexpr int kT = 16 * kTB;
  static constexpr bool kTwo = kTB >= 3;
  static constexpr int kStride = kT + 4;                 // row of A or B, elements
  static constexpr size_t kRows = (size_t)kT * Op::kRowBytes;
  static constexpr size_t kMat = (size_t)kT * kStride * 4;
  static constexpr size_t kDiag = (size_t)kTB * 16 * 20 * 4;
  static constexpr size_t kTail = 2 * kMat + 2 * kDiag;
  // A, B, diagonal blocks and inverses; kDeep: after two planes and the rows of one block
  static constexpr size_t kTailAt = kDeep ? 2 * kRows + 32 * Op::kRowBytes : kTwo ? 0 : 3 * kRows;
  static constexpr size_t kBytes = !kDeep && kTwo ? 2 * kRows : kTailAt + kTail;
  static_assert(!kTwo || kTail <= 2 * kRows, "matrices lie inside the planes");
};

// kDeep: A and B with the decays of each block of rows referred to its own R
// (64-node chains, floor -5, 64 x 32 heads: 379 to 389 us; pair by pair 3037).
template <int kTB, int kWaves, typename TIn, bool kDeep>
__global__ __launch_bounds__(64 * kWaves, kDeep ? 2 : 4) void tree_tile_kernel(
    const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
    const float* __restrict__ g, const float* __restrict__ beta, const float* __restrict__ state,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes, TIn* __restrict__ o, int H,
    int T, float scale, float g_min, uint32_t fe_flags, float fe_eps, int gate, int reach) {
  constexpr int D = 128;
  using Op = FloatOp;
  using L = TileLds<kTB, kDeep>;
  constexpr int kT = L::kT, kNT = 8 / kWaves;            // n-tiles of a wave
  const uint32_t n = blockIdx.x / (uint32_t)H, h = blockIdx.x % (uint32_t)H;
  const int nt = num_nodes ? min(max(num_nodes[n], 0), T) : T;
  if (nt == 0) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave), lane = tid % kWave;
  const int lr = lane % 16, lg = lane / 16;              // operand row / column, lane group
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* s_ke = lds;                                      // planes: k E, k / E, q E, [kT] rows each
  char* s_kq = s_ke + L::kRows;
  char* s_qe = L::kTwo || kDeep ? s_ke : s_kq + L::kRows;
  char* s_A = lds + L::kTailAt;                          // -beta A
  char* s_B = s_A + L::kMat;
  float* s_diag = (float*)(s_B + L::kMat);               // [kTB][16][20] diagonal blocks of -beta A
  char* s_inv = (char*)s_diag + L::kDiag;                // [kTB] 16 rows of stride 20
  __shared__ uint64_t s_anc[kMaxNodes];
  __shared__ __attribute__((aligned(16))) float s_b[kMaxNodes];
  __shared__ unsigned long long s_bad[2];                // nodes with d, with o not finite in every column
  __shared__ uint64_t s_gate[kWaves];                    // nodes with NaN decays in a wave's channels
  // Rows of this head inside the sequence by 32-bit byte offsets from uniform
  // bases (the launcher sees to 4 H D < 2^24): one instruction an address.
  const uint32_t row_bytes = (uint32_t)H * D * sizeof(TIn);
  const size_t first = ((size_t)n * T * H + h) * D;
  auto off = [&](int t) __attribute__((always_inline)) { return __umul24((uint32_t)t, row_bytes); };

  const int parent = lane < nt ? clean_parent(parents, (size_t)n * T, lane) : -1;
  const float braw = beta[((size_t)n * T + min(lane, nt - 1)) * H + h];
  // Lane (group, node) holds kC consecutive channels of its node; a wave all
  // nodes of 128 / kWaves channels, so that decays multiply along the paths by
  // exchanges inside the wave.
  constexpr int kNodes = kTB <= 2 ? kT : 64, kC = D / kWaves / (kWave / kNodes);
  const int node = lane % kNodes, chan = wave * (D / kWaves) + lane / kNodes * kC;
  const bool live = node < nt;
  Run<TIn, kC> lk, lq;
  float te[kC];
  {
    const uint32_t at = off(min(node, nt - 1)) + chan * (uint32_t)sizeof(TIn);
    lk.load((const char*)(k + first) + at);
    lq.load((const char*)(q + first) + at);
    if (gate == KDA_GATE_CHANNEL) {
      Run<float, kC> lg4;
      lg4.load((const char*)(g + first) + __umul24((uint32_t)min(node, nt - 1), (uint32_t)H * D * 4) + chan * 4u);
#pragma unroll
      for (int c = 0; c < kC; ++c) te[c] = lg4.get(c);
    } else {
      const float one = gate == KDA_GATE_HEAD ? g[((size_t)n * T + min(node, nt - 1)) * H + h] : 0.f;
#pragma unroll
      for (int c = 0; c < kC; ++c) te[c] = one;
    }
  }
  // S in operand layout: rows 32 ks + 8 lg + j, columns col0 + kNT lr + {0 ..}
  const int col0 = wave * 16 * kNT;
  // (a uniform base and one 32-bit lane offset: no 64-bit address per load).
  // With two n-tiles a wave reads whole 128-byte lines, once, past the caches
  // (256x32 heads, 16 nodes: 184 us, 185 through them); with one, two waves share them.
  const uint32_t lane_off = (uint32_t)(8 * lg * D + kNT * lr) * 4;
  float sreg[4][8][kNT];
  auto load_s = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const char* base = (const char*)(state + (size_t)blockIdx.x * D * D + col0 + 32 * ks * D) + lane_off;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int c = 0; c < kNT; ++c)
          sreg[ks][j][c] = kNT == 2 ? __builtin_nontemporal_load((const float*)base + j * D + c)
                                    : ((const float*)base)[j * D + c];
    }
  };
  if constexpr (!L::kTwo && !kDeep) load_s();
  const uint32_t cols = kNT * lr * sizeof(TIn);
  using Cols = std::conditional_t<kNT == 2, Pair<TIn>, One<TIn>>;
  Cols vreg[kTB][4];
  auto load_v = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int I = 0; I < kTB; ++I)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vreg[I][r].load((const TIn*)((const char*)(v + first + col0) + off(min(16 * I + 4 * lg + r, nt - 1)) + cols));
  };
  if constexpr (!L::kTwo && !kDeep) load_v();

  // the tree: ancestors, and whether this kernel takes it
  const uint64_t anc = ancestors(parent, lane);
  if (kDeep && block_depth(anc, lane < nt) > reach) return;   // the path kernel takes it
  if (wave == 0) {
    s_anc[lane] = anc;
    s_b[lane] = lane >= nt ? 0.f : fe_flags & KDA_FE_BETA_LOGITS ? beta_logit(braw) : braw;
    if (lane < 2) s_bad[lane] = 0;
  }
  // decays, normalised rows; a node with a NaN decay is remembered as bad, the
  // decay itself is the floor's from here on (the clamps drop NaN)
  bool nan_gate = false;
#pragma unroll
  for (int c = 0; c < kC; ++c) nan_gate |= te[c] != te[c];
  uint64_t nan_nodes = __ballot(nan_gate && live);
  if (kNodes <= 32) nan_nodes |= nan_nodes >> 32;
  if (kNodes == 16) nan_nodes |= nan_nodes >> 16;
  if (lane == 0) s_gate[wave] = nan_nodes & (~0ull >> (64 - kNodes));
  const float alpha_min = __builtin_amdgcn_exp2f(g_min * kLog2e);
  double G[kC];                                           // (kDeep)
  if constexpr (kDeep) {
#pragma unroll
    for (int c = 0; c < kC; ++c) G[c] = log2_alpha(te[c], fe_flags & KDA_FE_GATE_LOGITS, g_min);
  } else if (gate == KDA_GATE_NONE) {
#pragma unroll
    for (int c = 0; c < kC; ++c) te[c] = 1.f;
  } else if (fe_flags & KDA_FE_GATE_LOGITS) {
#pragma unroll
    for (int c = 0; c < kC; ++c) te[c] = gate_alpha_logit(te[c], alpha_min);
  } else {
#pragma unroll
    for (int c = 0; c < kC; ++c) te[c] = gate_alpha(te[c], g_min);
  }
  // scales of k and q: 1 or the inverse norms (sums over the waves by LDS)
  float rk = 1.f, rq = 1.f;
  if (fe_flags & KDA_FE_L2NORM_QK) {
    float sk = 0.f, sq = 0.f;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      sk += lk.get(c) * lk.get(c);
      sq += lq.get(c) * lq.get(c);
    }
#pragma unroll
    for (int m = kNodes; m < kWave; m *= 2) { sk += __shfl_xor(sk, m); sq += __shfl_xor(sq, m); }
    f32x2* s_norm = (f32x2*)lds;                          // [kWaves][kNodes]
    if (lane < kNodes) s_norm[wave * kNodes + node] = f32x2{sk, sq};
    lds_barrier();
    f32x2 sum = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += s_norm[w * kNodes + node];
    rk = inv_norm(sum[0], fe_eps);
    rq = inv_norm(sum[1], fe_eps);
    lds_barrier();                                        // the planes come over it
  }
  if constexpr (L::kTwo || kDeep) {      // behind q, k and g, which are needed first
    load_s();
    __builtin_amdgcn_sched_barrier(0);
  }
  // E by doubling: after r rounds the product over the last 2^r nodes of the path
  if (gate != KDA_GATE_NONE) {
    const int base = lane - node;
    for (int jump = __shfl(parent, node); __ballot(jump >= 0);) {
      const int from = base + max(jump, 0);
      const int next = __shfl(jump, from);
      if constexpr (kDeep) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const double e = __shfl(G[c], from);
          G[c] += jump >= 0 ? e : 0.0;
        }
      } else {
        float e[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) e[c] = __shfl(te[c], from);
#pragma unroll
        for (int c = 0; c < kC; ++c) te[c] *= jump >= 0 ? e[c] : 1.f;
      }
      jump = jump >= 0 ? next : -1;
    }
  }
  if constexpr (kDeep) {
#pragma unroll
    for (int c = 0; c < kC; ++c) te[c] = exp2_wide(G[c]);
  }
  // rows past the last node are 0
  auto put_q = [&]() __attribute__((always_inline)) {
    float x[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) x[c] = live ? lq.get(c) * rq * te[c] : 0.f;
    if (kNodes == kT || node < kT) Op::put(s_qe + node * Op::kRowBytes, chan, x);
  };
  {
    float x[kC], y[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const float kc = live ? lk.get(c) * rk : 0.f;
      x[c] = kc * te[c];
      y[c] = live && !kDeep ? kc * __builtin_amdgcn_rcpf(te[c]) : 0.f;
    }
    if (kNodes == kT || node < kT) {
      Op::put(s_ke + node * Op::kRowBytes, chan, x);
      if (!kDeep) Op::put(s_kq + node * Op::kRowBytes, chan, y);
    }
  }
  if constexpr (!L::kTwo && !kDeep) put_q();
  lds_barrier();

  // U = (k E) S and W = (q E) S; A and B by tiles (I, J <= I), shared out over
  // the waves. Units of tiles: A and B alternate, or (kTwo) A's, then B's.
  constexpr int kPairs = kTB * (kTB + 1) / 2;
  constexpr int kTurns = L::kTwo ? (kPairs + kWaves - 1) / kWaves : (2 * kPairs + kWaves - 1) / kWaves;
  constexpr int kSets = L::kTwo ? 2 : 1;
  f32x4 mat[kSets][kTurns];
  auto tile_of = [&](int set, int turn, bool& is_b, int& I, int& J) __attribute__((always_inline)) {
    const int unit = wave + kWaves * turn, pair = L::kTwo ? unit : unit >> 1;
    is_b = L::kTwo ? set == 1 : unit & 1;
    I = (pair >= 1) + (pair >= 3) + (pair >= 6);
    J = pair - I * (I + 1) / 2;
    return pair < kPairs;
  };
  auto tiles = [&](auto Set) __attribute__((always_inline)) {
    constexpr int set = decltype(Set)::value;
    static_for<0, kTurns>([&](auto X) __attribute__((always_inline)) {
      constexpr int x = decltype(X)::value;
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
      bool is_b;
      int I, J;
      if (tile_of(set, x, is_b, I, J)) {
        const char* rows = is_b ? s_qe : s_ke;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          y = Op::mma(Op::get8(rows + (16 * I + lr) * Op::kRowBytes, 32 * ks + 8 * lg),
                      Op::get8(s_kq + (16 * J + lr) * Op::kRowBytes, 32 * ks + 8 * lg), y);
      }
      mat[set][x] = y;
    });
  };
  f32x4 U[kTB][kNT], W[kTB][kNT];
#pragma unroll
  for (int I = 0; I < kTB; ++I)
#pragma unroll
    for (int c = 0; c < kNT; ++c) U[I][c] = W[I][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  typename Op::F8 sf[4][kNT];              // S as operands, in place of sreg
  auto times_s = [&](bool u, bool w) __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (u) {
#pragma unroll
        for (int c = 0; c < kNT; ++c) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = sreg[ks][j][c];
          sf[ks][c] = Op::make8(x);
        }
      }
#pragma unroll
      for (int I = 0; I < kTB; ++I) {
        if (u) {
          const typename Op::F8 a = Op::get8(s_ke + (16 * I + lr) * Op::kRowBytes, 32 * ks + 8 * lg);
#pragma unroll
          for (int c = 0; c < kNT; ++c) U[I][c] = Op::mma(a, sf[ks][c], U[I][c]);
        }
        if (w) {
          const typename Op::F8 a = Op::get8(s_qe + (16 * I + lr) * Op::kRowBytes, 32 * ks + 8 * lg);
#pragma unroll
          for (int c = 0; c < kNT; ++c) W[I][c] = Op::mma(a, sf[ks][c], W[I][c]);
        }
      }
    }
  };
  // a tile of A or B, masked to ancestors, to LDS
  auto put_tile = [&](bool is_b, int I, int J, f32x4 m) __attribute__((always_inline)) {
    const int j = 16 * J + lr;
    const uint32_t* anc32 = (const uint32_t*)s_anc + (J >> 1);
    f32x4 y;
    bool odd = false;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * I + 4 * lg + r;
      const bool on = (anc32[2 * i] >> (j & 31) & 1) && (is_b || i != j);
      y[r] = on ? (is_b ? m[r] : -s_b[i] * m[r]) : 0.f;
      odd |= !is_finite(y[r]);
    }
    if (__ballot(odd)) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!is_finite(y[r])) {
          atomicOr(&s_bad[is_b], 1ull << (16 * I + 4 * lg + r));
          y[r] = 0.f;
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      Op::put1(is_b ? s_B : s_A, L::kStride, 16 * I + 4 * lg + r, j, y[r]);
      if (!is_b && I == J) s_diag[(16 * I + 4 * lg + r) * 20 + lr] = y[r];
    }
  };
  if constexpr (kDeep) {
    times_s(true, false);
    lds_barrier();
    put_q();
    lds_barrier();
    times_s(false, true);
    load_v();
    static_for<0, kTB>([&](auto II) __attribute__((always_inline)) {
      constexpr int I = decltype(II)::value;
      if (16 * I < nt) {
        char* s_rows = s_kq + L::kRows;                     // 16 rows of k, 16 of q
        const bool mine = node / 16 == I;
        float x[kC], y[kC], z[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          float hi = live ? (float)G[c] : -__builtin_inff(), lo = live ? (float)G[c] : __builtin_inff();
          hi = fmaxf(hi, row_ror<8>(hi)); hi = fmaxf(hi, row_ror<4>(hi));
          hi = fmaxf(hi, row_ror<2>(hi)); hi = fmaxf(hi, row_ror<1>(hi));
          lo = fminf(lo, row_ror<8>(lo)); lo = fminf(lo, row_ror<4>(lo));
          lo = fminf(lo, row_ror<2>(lo)); lo = fminf(lo, row_ror<1>(lo));
          const double R = (double)__shfl(0.5f * (hi + lo), lane - node + 16 * I);
          const float kc = live ? lk.get(c) * rk : 0.f, e = exp2_wide(G[c] - R);
          // (2^(R - G) may overflow for nodes that are nobody's ancestor here)
          x[c] = live ? kc * e : 0.f;
          y[c] = live ? lq.get(c) * rq * e : 0.f;
          z[c] = live ? kc * exp2_wide(R - G[c]) : 0.f;
        }
        if (mine) {
          Op::put(s_rows + (node % 16) * Op::kRowBytes, chan, x);
          Op::put(s_rows + (16 + node % 16) * Op::kRowBytes, chan, y);
        }
        if (node < 16 * (I + 1)) Op::put(s_kq + node * Op::kRowBytes, chan, z);
        lds_barrier();
        static_for<0, (2 * (I + 1) + kWaves - 1) / kWaves>([&](auto X) __attribute__((always_inline)) {
          const int unit = wave + kWaves * decltype(X)::value, J = unit >> 1;
          if (J <= I) {
            const bool is_b = unit & 1;
            f32x4 m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              m = Op::mma(Op::get8(s_rows + (16 * is_b + lr) * Op::kRowBytes, 32 * ks + 8 * lg),
                          Op::get8(s_kq + (16 * J + lr) * Op::kRowBytes, 32 * ks + 8 * lg), m);
            put_tile(is_b, I, J, m);
          }
        });
        lds_barrier();
      }
    });
  } else if constexpr (L::kTwo) {
    tiles(std::integral_constant<int, 0>{});
    times_s(true, false);
    lds_barrier();
    put_q();
    lds_barrier();
    tiles(std::integral_constant<int, 1>{});
    times_s(false, true);
    load_v();                              // (no registers to spare for it before)
    lds_barrier();
  } else {
    tiles(std::integral_constant<int, 0>{});
    times_s(true, true);
  }
  if constexpr (!kDeep)
    static_for<0, kSets * kTurns>([&](auto X) __attribute__((always_inline)) {
      constexpr int set = decltype(X)::value / kTurns, x = decltype(X)::value % kTurns;
      bool is_b;
      int I, J;
      if (tile_of(set, x, is_b, I, J)) put_tile(is_b, I, J, mat[set][x]);
    });
  lds_barrier();

  // Inverses X of I + beta A = I - N on the diagonal blocks, row lr of block lg
  // in lane (lg, lr), last column first: X = I + X N, so
  // x_j = (j == lr) + sum_{i > j} x_i N_ij, with N_ij broadcast from lane j of
  // its row of lanes. (Substitution: powers of N would lose digits where keys repeat.)
  f32x4 inv = {0.f, 0.f, 0.f, 0.f};                       // kTB = 1: X[lr][4 lg ..]
  if (kTB == 1 || wave == 0) {
    const float* m = s_diag + (kTB == 1 ? 0 : min(lg, kTB - 1)) * 16 * 20 + lr;
    float nr[16], x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) nr[i] = m[i * 20];
    static_for<0, 16>([&](auto JJ) __attribute__((always_inline)) {
      constexpr int j = 15 - decltype(JJ)::value;
      float s0 = j == lr ? 1.f : 0.f, s1 = 0.f;
      static_for<j + 1, 16>([&](auto I) __attribute__((always_inline)) {
        constexpr int i = decltype(I)::value;
        // the newest x last, so that it is waited for last
        if constexpr ((i - j) % 2) s1 += row_bcast<j>(nr[16 + j - i]) * x[16 + j - i];
        else s0 += row_bcast<j>(nr[16 + j - i]) * x[16 + j - i];
      });
      x[j] = s0 + s1;
      // formed here: the compiler would move the sums to their use and leave all
      // 120 broadcasts in registers until then
      asm volatile("" : "+v"(x[j]));
    });
    if constexpr (kTB == 1) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        inv[r] = lg < 2 ? (lg == 0 ? x[r] : x[4 + r]) : (lg == 2 ? x[8 + r] : x[12 + r]);
    } else if (lg < kTB) {
#pragma unroll
      for (int j = 0; j < 16; ++j) Op::put1(s_inv, 20, 16 * lg + lr, j, x[j]);
    }
  }
  if constexpr (kTB > 1) lds_barrier();

  // d and o, block by block; bit 16 I + 4 lg + r of bad[c]: that row of the
  // lane's column is not finite
  typename Op::F4 d[kTB][kNT];
  uint64_t bad[kNT] = {};
  auto clean = [&](f32x4& x, int I, int c) __attribute__((always_inline)) {
    if (__ballot(!(is_finite(x[0]) && is_finite(x[1]) && is_finite(x[2]) && is_finite(x[3])))) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!is_finite(x[r])) {
          bad[c] |= 1ull << (16 * I + 4 * lg + r);
          x[r] = 0.f;
        }
    }
  };
#pragma unroll
  for (int I = 0; I < kTB; ++I) {
    if (16 * I < nt) {
      const f32x4 b4 = *(const f32x4*)(s_b + 16 * I + 4 * lg);
#pragma unroll
      for (int c = 0; c < kNT; ++c) {
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          x[r] = 16 * I + 4 * lg + r < nt ? b4[r] * (vreg[I][r].get(c) - U[I][c][r]) : 0.f;
#pragma unroll
        for (int J = 0; J < I; ++J)
          x = Op::mma(Op::get4(s_A, L::kStride, 16 * I + lr, 16 * J + 4 * lg), d[J][c], x);
        clean(x, I, c);
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        typename Op::F4 a;
        if constexpr (kTB == 1) a = Op::make4(inv);
        else a = Op::get4(s_inv, 20, 16 * I + lr, 4 * lg);
        y = Op::mma(a, Op::make4(x), y);
        clean(y, I, c);
        d[I][c] = Op::make4(y);
      }
    }
  }
  uint64_t bad_d = s_bad[0], bad_o = s_bad[1];
#pragma unroll
  for (int w = 0; w < kWaves; ++w) bad_d |= s_gate[w];
  bool any = bad_d | bad_o;
#pragma unroll
  for (int c = 0; c < kNT; ++c) any |= bad[c] != 0;
  any = __ballot(any) != 0;
  if (any) {
#pragma unroll
    for (int c = 0; c < kNT; ++c) {
      bad[c] |= __shfl_xor((unsigned long long)bad[c], 16);
      bad[c] |= __shfl_xor((unsigned long long)bad[c], 32);
      bad[c] |= bad_d;
    }
  }
#pragma unroll
  for (int I = 0; I < kTB; ++I) {
    if (16 * I < nt) {
#pragma unroll
      for (int c = 0; c < kNT; ++c)
#pragma unroll
        for (int J = 0; J <= I; ++J)
          W[I][c] = Op::mma(Op::get4(s_B, L::kStride, 16 * I + lr, 16 * J + 4 * lg), d[J][c], W[I][c]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * I + 4 * lg + r;
        if (i < nt) {
          float y[kNT];
#pragma unroll
          for (int c = 0; c < kNT; ++c) {
            y[c] = scale * W[I][c][r];
            if (any && ((s_anc[i] & bad[c]) || (bad_o >> i & 1))) y[c] = __builtin_nanf("");
          }
          Cols::store((TIn*)((char*)(o + first + col0) + off(i) + cols), y[0], y[kNT - 1]);
        }
      }
    }
  }
}

// ---- D = 16 --------------------------------------------------------------------------
// The same blocks of 16 nodes, one wave per head and no LDS: lane (group lg, lr)
// holds channels 4 lg .. + 3 of node 16 I + lr, which is the operand layout of
// a 16 x 16 x 16 product, and A and B are formed transposed, which leaves them
// in operand layout too. All products are fp32 (16 x 16 x 4). The decays always
// have their block's reference. 64 x 32 heads, chains of 64 nodes: 40 us, bound
// by the chain of dependent instructions of a wave (pair by pair 838 us).
template <int kTB, typename TIn>
__global__ __launch_bounds__(256, kTB >= 3 ? 2 : 4) void tree_small_kernel(
    const TIn* __restrict__ q, const TIn* __restrict__ k, const TIn* __restrict__ v,
    const float* __restrict__ g, const float* __restrict__ beta, const float* __restrict__ state,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes, TIn* __restrict__ o,
    uint32_t heads, int H, int T, float scale, float g_min, uint32_t fe_flags, float fe_eps, int gate, int reach) {
  constexpr int D = 16;
  using Op = FloatOp;
  const uint32_t head = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (head >= heads) return;
  const uint32_t n = head / (uint32_t)H, h = head % (uint32_t)H;
  const int nt = num_nodes ? min(max(num_nodes[n], 0), T) : T;
  if (nt == 0) return;
  const int lane = threadIdx.x % kWave, lr = lane % 16, lg = lane / 16;
  auto row = [&](int t) __attribute__((always_inline)) { return ((size_t)n * T + t) * H + h; };
  const int parent = lane < nt ? clean_parent(parents, (size_t)n * T, lane) : -1;
  const float braw = beta[row(min(lane, nt - 1))];
  float kv[kTB][4], qv[kTB][4], gv[kTB][4];
#pragma unroll
  for (int I = 0; I < kTB; ++I) {
    const size_t at = row(min(16 * I + lr, nt - 1));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      kv[I][c] = Elem<TIn>::load(k + at * D + 4 * lg + c);
      qv[I][c] = Elem<TIn>::load(q + at * D + 4 * lg + c);
      gv[I][c] = gate == KDA_GATE_NONE ? 0.f : g[gate == KDA_GATE_CHANNEL ? at * D + 4 * lg + c : at];
    }
  }
  Op::F4 sf;                                   // S[4 lg + j][lr]
#pragma unroll
  for (int j = 0; j < 4; ++j) sf.x[j] = state[(size_t)head * D * D + (4 * lg + j) * D + lr];
  float vv[kTB][4];
#pragma unroll
  for (int I = 0; I < kTB; ++I)
#pragma unroll
    for (int r = 0; r < 4; ++r) vv[I][r] = Elem<TIn>::load(v + row(min(16 * I + 4 * lg + r, nt - 1)) * D + lr);

  const uint64_t anc = ancestors(parent, lane);
  if (block_depth(anc, lane < nt) > reach) return;          // the path kernel takes it
  const float b = fe_flags & KDA_FE_BETA_LOGITS ? beta_logit(braw) : braw;
  if (fe_flags & KDA_FE_L2NORM_QK) {
#pragma unroll
    for (int I = 0; I < kTB; ++I) {
      float sk = 0.f, sq = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) { sk += kv[I][c] * kv[I][c]; sq += qv[I][c] * qv[I][c]; }
      sk += __shfl_xor(sk, 16); sk += __shfl_xor(sk, 32);
      sq += __shfl_xor(sq, 16); sq += __shfl_xor(sq, 32);
      const float rk = inv_norm(sk, fe_eps), rq = inv_norm(sq, fe_eps);
#pragma unroll
      for (int c = 0; c < 4; ++c) { kv[I][c] *= rk; qv[I][c] *= rq; }
    }
  }
  // G by doubling inside each block, then on from the path's last node before it
  uint64_t bad_d = 0, bad_o = 0;             // nodes with d, with o not finite in every column
  double G[kTB][4];
  static_for<0, kTB>([&](auto II) __attribute__((always_inline)) {
    constexpr int I = decltype(II)::value;
    const bool live = 16 * I + lr < nt;
    bool odd = false;                        // a NaN decay, which log2_alpha's clamps drop
#pragma unroll
    for (int c = 0; c < 4; ++c) odd |= gv[I][c] != gv[I][c];
    uint64_t m = __ballot(odd && live);
    m |= m >> 32;
    m |= m >> 16;
    bad_d |= (m & 0xffff) << (16 * I);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!live) kv[I][c] = qv[I][c] = 0.f;
      G[I][c] = gate == KDA_GATE_NONE ? 0.0 : log2_alpha(gv[I][c], fe_flags & KDA_FE_GATE_LOGITS, g_min);
    }
    int up = __shfl(parent, 16 * I + lr);
    while (__ballot(up >= 16 * I)) {
      const int from = 16 * lg + (up & 15);
      const bool on = up >= 16 * I;
      const int next = __shfl(up, from);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const double x = __shfl(G[I][c], from);
        G[I][c] += on ? x : 0.0;
      }
      up = on ? next : up;
    }
    static_for<0, I>([&](auto JJ) __attribute__((always_inline)) {
      constexpr int J = decltype(JJ)::value;
      const bool on = up >= 0 && up / 16 == J;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const double x = __shfl(G[J][c], 16 * lg + (up & 15));
        G[I][c] += on ? x : 0.0;
      }
    });
  });

  // U, W, A and B (transposed products: acc[r] = element (row lr, column 4 lg + r))
  f32x4 U[kTB], W[kTB], A[kTB][kTB], B[kTB][kTB];
  auto note = [&](f32x4& x, int I, uint64_t& bits) __attribute__((always_inline)) {
    const bool odd = !(is_finite(x[0]) && is_finite(x[1]) && is_finite(x[2]) && is_finite(x[3]));
    uint64_t m = __ballot(odd);
    if (m) {
      m |= m >> 32;
      m |= m >> 16;
      bits |= (m & 0xffff) << (16 * I);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = is_finite(x[r]) ? x[r] : 0.f;
    }
  };
  static_for<0, kTB>([&](auto II) __attribute__((always_inline)) {
    constexpr int I = decltype(II)::value;
    U[I] = W[I] = f32x4{0.f, 0.f, 0.f, 0.f};
    static_for<0, I + 1>([&](auto JJ) __attribute__((always_inline)) {
      A[I][decltype(JJ)::value] = B[I][decltype(JJ)::value] = f32x4{0.f, 0.f, 0.f, 0.f};
    });
    if (16 * I < nt) {
      const bool live = 16 * I + lr < nt;
      Op::F4 ke, qe, kr, qr;
      double R[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float hi = live ? (float)G[I][c] : -__builtin_inff(), lo = live ? (float)G[I][c] : __builtin_inff();
        hi = fmaxf(hi, row_ror<8>(hi)); hi = fmaxf(hi, row_ror<4>(hi));
        hi = fmaxf(hi, row_ror<2>(hi)); hi = fmaxf(hi, row_ror<1>(hi));
        lo = fminf(lo, row_ror<8>(lo)); lo = fminf(lo, row_ror<4>(lo));
        lo = fminf(lo, row_ror<2>(lo)); lo = fminf(lo, row_ror<1>(lo));
        R[c] = 0.5 * ((double)hi + (double)lo);
        const float e = exp2_wide(G[I][c]), er = live ? exp2_wide(G[I][c] - R[c]) : 0.f;
        ke.x[c] = kv[I][c] * e;
        qe.x[c] = qv[I][c] * e;
        kr.x[c] = kv[I][c] * er;
        qr.x[c] = qv[I][c] * er;
      }
      U[I] = Op::mma(ke, sf, U[I]);
      W[I] = Op::mma(qe, sf, W[I]);
      const uint64_t mine = __shfl((unsigned long long)anc, 16 * I + lr);
      const float bi = -__shfl(b, 16 * I + lr);
      static_for<0, I + 1>([&](auto JJ) __attribute__((always_inline)) {
        constexpr int J = decltype(JJ)::value;
        Op::F4 kq;
#pragma unroll
        for (int c = 0; c < 4; ++c) kq.x[c] = kv[J][c] * exp2_wide(R[c] - G[J][c]);
        f32x4 a = {0.f, 0.f, 0.f, 0.f}, bb = {0.f, 0.f, 0.f, 0.f};
        a = Op::mma(kq, kr, a);
        bb = Op::mma(kq, qr, bb);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * J + 4 * lg + r;
          const bool on = live && (mine >> j & 1);
          a[r] = on && j != 16 * I + lr ? bi * a[r] : 0.f;
          bb[r] = on ? bb[r] : 0.f;
        }
        note(a, I, bad_d);
        note(bb, I, bad_o);
        A[I][J] = a;
        B[I][J] = bb;
      });
    }
  });

  // d and o, block by block
  Op::F4 d[kTB];
  uint64_t bad = 0;                           // rows of the lane's column that are not finite
  auto clean = [&](f32x4& x, int I) __attribute__((always_inline)) {
    if (__ballot(!(is_finite(x[0]) && is_finite(x[1]) && is_finite(x[2]) && is_finite(x[3])))) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (!is_finite(x[r])) {
          bad |= 1ull << (16 * I + 4 * lg + r);
          x[r] = 0.f;
        }
    }
  };
  static_for<0, kTB>([&](auto II) __attribute__((always_inline)) {
    constexpr int I = decltype(II)::value;
    d[I].x = f32x4{0.f, 0.f, 0.f, 0.f};
    if (16 * I < nt) {
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float bi = __shfl(b, 16 * I + 4 * lg + r);
        x[r] = 16 * I + 4 * lg + r < nt ? bi * (vv[I][r] - U[I][r]) : 0.f;
      }
      static_for<0, I>([&](auto JJ) __attribute__((always_inline)) {
        constexpr int J = decltype(JJ)::value;
        x = Op::mma(Op::F4{A[I][J]}, d[J], x);
      });
      clean(x, I);
      // (I - N)^-1 X by substitution: row lr of the inverse, last column first,
      // N_ij from lane (j / 4, i)
      float y[16];
      static_for<0, 16>([&](auto C) __attribute__((always_inline)) {
        constexpr int j = 15 - decltype(C)::value;
        float s0 = j == lr ? 1.f : 0.f;
        static_for<j + 1, 16>([&](auto K) __attribute__((always_inline)) {
          constexpr int i = 16 + j - decltype(K)::value;
          s0 += y[i] * __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, (float)A[I][I][j % 4]),
                                                                          j / 4 * 16 + i));
        });
        y[j] = s0;
        asm volatile("" : "+v"(y[j]));
      });
      f32x4 inv;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        inv[r] = lg < 2 ? (lg == 0 ? y[r] : y[4 + r]) : (lg == 2 ? y[8 + r] : y[12 + r]);
      f32x4 z = {0.f, 0.f, 0.f, 0.f};
      z = Op::mma(Op::F4{inv}, Op::make4(x), z);
      clean(z, I);
      d[I].x = z;
    }
  });
  const bool any = __ballot(bad != 0) || bad_d || bad_o;
  if (any) {
    bad |= __shfl_xor((unsigned long long)bad, 16);
    bad |= __shfl_xor((unsigned long long)bad, 32);
    bad |= bad_d;
  }
  static_for<0, kTB>([&](auto II) __attribute__((always_inline)) {
    constexpr int I = decltype(II)::value;
    if (16 * I < nt) {
      f32x4 y = W[I];
      static_for<0, I + 1>([&](auto JJ) __attribute__((always_inline)) {
        constexpr int J = decltype(JJ)::value;
        y = Op::mma(Op::F4{B[I][J]}, d[J], y);
      });
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * I + 4 * lg + r;
        float out = scale * y[r];
        if (any) {
          const uint64_t mine = __shfl((unsigned long long)anc, i);
          if ((mine & bad) || (bad_o >> i & 1)) out = __builtin_nanf("");
        }
        if (i < nt) Elem<TIn>::store(o + row(i) * D + lr, out);
      }
    }
  });
}

template <int D, typename TIn>
static hipError_t launch_paths(const TreeArgs& a, int taken) {
  const unsigned blocks = (unsigned)((int64_t)a.N * a.H);
  hipLaunchKernelGGL((tree_path_kernel<D, TIn>), dim3(blocks), dim3(256), path_lds_bytes<D>(a.T), a.stream,
                     (const TIn*)a.q, (const TIn*)a.k, (const TIn*)a.v, a.g, a.beta, a.state, a.parents,
                     a.num_nodes, (TIn*)a.o, a.H, a.T, a.scale, a.g_min, a.fe_flags, a.fe_eps, (int)a.gate,
                     taken);
  return hipGetLastError();
}

template <int kTB, int kWaves, typename TIn, bool kDeep>
static hipError_t launch_tiles(const TreeArgs& a, int reach) {
  const unsigned blocks = (unsigned)((int64_t)a.N * a.H);
  constexpr size_t lds = TileLds<kTB, kDeep>::kBytes;
  static_assert(64 * kWaves <= (kTB == 1 ? kHeadThreads : kLargeTreeThreads), "threads that the launch limits count");
  hipLaunchKernelGGL((tree_tile_kernel<kTB, kWaves, TIn, kDeep>), dim3(blocks), dim3(64 * kWaves), lds, a.stream,
                     (const TIn*)a.q, (const TIn*)a.k, (const TIn*)a.v, a.g, a.beta, a.state, a.parents, a.num_nodes, (TIn*)a.o, a.H, a.T, a.scale, a.g_min, a.fe_flags,
                     a.fe_eps, (int)a.gate, reach);
  return hipGetLastError();
}

template <typename TIn, bool kDeep>
static hipError_t launch_blocks(const TreeArgs& a, int reach) {
  switch ((a.T + 15) / 16) {
    case 1: return launch_tiles<1, 4, TIn, kDeep>(a, reach);
    case 2: return launch_tiles<2, 8, TIn, kDeep>(a, reach);
    case 3: return launch_tiles<3, 8, TIn, kDeep>(a, reach);
    default: return launch_tiles<4, 8, TIn, kDeep>(a, reach);
  }
}

template <typename TIn>
static hipError_t launch_tree_128(const TreeArgs& a) {
  const int reach = reach_of(kMaxSpread, a.g_min, a.gate);
  // (the tile kernels' 24-bit row offsets: H D < 2^22)
  if (reach < 1 || (int64_t)a.H * 128 * 4 >= 1 << 24) return launch_paths<128, TIn>(a, kNoneTaken);
  if (reach_of(kMaxSpan, a.g_min, a.gate) >= a.T) return launch_blocks<TIn, false>(a, 0);
  const hipError_t e = launch_blocks<TIn, true>(a, reach);
  // (a block is at most T decays deep)
  if (e != hipSuccess || reach >= a.T) return e;
  return launch_paths<128, TIn>(a, reach);
}

template <int kTB, typename TIn>
static hipError_t launch_small(const TreeArgs& a, int reach) {
  const unsigned heads = (unsigned)((int64_t)a.N * a.H);
  hipLaunchKernelGGL((tree_small_kernel<kTB, TIn>), dim3(heads / 4 + (heads % 4 != 0)), dim3(256), 0, a.stream,
                     (const TIn*)a.q, (const TIn*)a.k, (const TIn*)a.v, a.g, a.beta, a.state, a.parents, a.num_nodes,
                     (TIn*)a.o, heads, a.H, a.T, a.scale, a.g_min, a.fe_flags, a.fe_eps, (int)a.gate, reach);
  return hipGetLastError();
}

template <typename TIn>
static hipError_t launch_tree_16(const TreeArgs& a) {
  const int reach = reach_of(kMaxSpread, a.g_min, a.gate);
  if (reach < 1) return launch_paths<16, TIn>(a, kNoneTaken);
  hipError_t e;
  switch ((a.T + 15) / 16) {
    case 1: e = launch_small<1, TIn>(a, reach); break;
    case 2: e = launch_small<2, TIn>(a, reach); break;
    case 3: e = launch_small<3, TIn>(a, reach); break;
    default: e = launch_small<4, TIn>(a, reach);
  }
  // (a block is at most T decays deep)
  if (e != hipSuccess || reach >= a.T) return e;
  return launch_paths<16, TIn>(a, reach);
}

hipError_t launch_tree(const TreeArgs& a) {
  if (a.D == 128) return a.bf16 ? launch_tree_128<bf16_bits>(a) : launch_tree_128<float>(a);
  return a.bf16 ? launch_tree_16<bf16_bits>(a) : launch_tree_16<float>(a);
}

// ---- commit of a path -------------------------------------------------------------
// The recurrence over the accepted nodes, the state in registers from its one
// read to its one write (8 D^2 bytes per head, which is what the call costs:
// 256 x 32 heads with paths of 0 to 16 nodes 206 to 222 us, 4.9 to 5.2 TB/s; up
// to eight nodes each take what a decode step does in the same loop over three
// sets of states, 219 to 231 us against 218, and 16 nodes 269).
// Thread layout as the decode kernel's: D = 128, a 256-thread workgroup per
// head, lane l of wave w owns columns 32w + 4(l % 8) .. +3 of rows
// (l / 8) + 8i; D = 16, one wave per head.
// The nodes' vectors are staged kBatch nodes at a time; the first batch is
// loaded ahead of the state so that both are in flight together (behind it
// measured the same).
constexpr int kBatch = 8;

template <int D, typename TIn>
__global__ __launch_bounds__(D == 128 ? 256 : 64) void commit_kernel(
    const TIn* __restrict__ k, const TIn* __restrict__ v, const float* __restrict__ g,
    const float* __restrict__ beta, float* __restrict__ state, const int32_t* __restrict__ path,
    const int32_t* __restrict__ accept, int H, int T, float g_min, uint32_t fe_flags, float fe_eps, int gate) {
  constexpr int kThreads = D == 128 ? 256 : 64;
  constexpr int kColGroups = D == 128 ? 8 : 4;
  constexpr int kRowGroups = kWave / kColGroups;
  constexpr int kRowsPerLane = D / kRowGroups;
  constexpr int kRowSteps = D == 128 ? 3 : 4;
  constexpr int kIters = kBatch * D / kThreads;
  const uint32_t head = blockIdx.x, n = head / (uint32_t)H, h = head % (uint32_t)H;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
  const int cg = lane % kColGroups, rg = lane / kColGroups;
  const int col = wave * 4 * kColGroups + 4 * cg;
  int len = min(max(accept[n], 0), T);
  if (len == 0) return;
  const int node_of_lane = path[(size_t)n * T + min(lane, T - 1)];
  // the path's length: accept, cut before the first index outside [0, T)
  const uint64_t bad = __ballot(!(lane < T && node_of_lane >= 0 && node_of_lane < T));
  if (bad) len = min(len, __builtin_ctzll(bad));
  if (len == 0) return;
  // row of the path's node i; called by all lanes together (it reads lane i)
  auto row = [&](int i) __attribute__((always_inline)) {
    return ((size_t)n * T + __builtin_amdgcn_ds_bpermute(4 * i, node_of_lane)) * H + h;
  };
  const float alpha_min = __builtin_amdgcn_exp2f(g_min * kLog2e);
  const bool norm = fe_flags & KDA_FE_L2NORM_QK;

  __shared__ float s_k[kBatch][D], s_a[kBatch][D], s_v[kBatch][D], s_b[kBatch];
  float tk[kIters], ta[kIters], tv[kIters], tb = 0.f;
  // element e = t * D + c of a batch, clamped into the path
  auto fetch = [&](int first) __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < kIters; ++x) {
      const int e = tid + x * kThreads, c = e % D;
      const size_t r = row(min(first + e / D, len - 1));
      tk[x] = Elem<TIn>::load(k + r * D + c);
      tv[x] = Elem<TIn>::load(v + r * D + c);
      ta[x] = gate == KDA_GATE_NONE ? 0.f : g[gate == KDA_GATE_CHANNEL ? r * D + c : r];
    }
    tb = beta[row(min(first + tid % kBatch, len - 1))];
  };
  auto stage = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < kIters; ++x) {
      const int e = tid + x * kThreads, t = e / D, c = e % D;
      s_k[t][c] = tk[x];
      s_v[t][c] = tv[x];
      s_a[t][c] = gate == KDA_GATE_NONE            ? 1.f
                  : ta[x] != ta[x]                ? ta[x]        // (the clamps would drop a NaN)
                  : fe_flags & KDA_FE_GATE_LOGITS ? gate_alpha_logit(ta[x], alpha_min)
                                                  : gate_alpha(ta[x], g_min);
    }
    if (tid < kBatch) s_b[tid] = fe_flags & KDA_FE_BETA_LOGITS ? beta_logit(tb) : tb;
  };
  fetch(0);
  float* S = state + (size_t)head * D * D;
  f32x4 s[kRowsPerLane];
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i) s[i] = *(const f32x4*)(S + (size_t)(rg + kRowGroups * i) * D + col);
  stage();
  lds_barrier();
  for (int first = 0;;) {
    const int cnt = min(kBatch, len - first);
    for (int t = 0; t < cnt; ++t) {
      f32x4 u = {0.f, 0.f, 0.f, 0.f};
      float kk = 0.f;
#pragma unroll
      for (int i = 0; i < kRowsPerLane; ++i) {
        const int r = rg + kRowGroups * i;
        const float kr = s_k[t][r];
        s[i] *= s_a[t][r];
        u += s[i] * kr;
        kk += kr * kr;
      }
      static_for<0, kRowSteps>([&](auto I) __attribute__((always_inline)) {
        constexpr int m = kColGroups << decltype(I)::value;
#pragma unroll
        for (int c = 0; c < 4; ++c) u[c] += lane_xor<m>(u[c]);
        kk += lane_xor<m>(kk);
      });
      const float rk = norm ? inv_norm(kk, fe_eps) : 1.f;
      const f32x4 d = (s_b[t] * rk) * (*(const f32x4*)&s_v[t][col] - u * rk);
#pragma unroll
      for (int i = 0; i < kRowsPerLane; ++i) s[i] += s_k[t][rg + kRowGroups * i] * d;
    }
    first += cnt;
    if (first >= len) break;
    fetch(first);
    __syncthreads();
    stage();
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kRowsPerLane; ++i)
    __builtin_nontemporal_store(s[i], (f32x4*)(S + (size_t)(rg + kRowGroups * i) * D + col));
}

template <int D, typename TIn>
static hipError_t launch_commit_t(const TreeArgs& a) {
  const unsigned blocks = (unsigned)((int64_t)a.N * a.H);
  hipLaunchKernelGGL((commit_kernel<D, TIn>), dim3(blocks), dim3(D == 128 ? 256 : 64), 0, a.stream,
                     (const TIn*)a.k, (const TIn*)a.v, a.g, a.beta, a.state, a.path, a.accept, a.H, a.T, a.g_min,
                     a.fe_flags, a.fe_eps, (int)a.gate);
  return hipGetLastError();
}

hipError_t launch_commit(const TreeArgs& a) {
  if (a.D == 128) return a.bf16 ? launch_commit_t<128, bf16_bits>(a) : launch_commit_t<128, float>(a);
  return a.bf16 ? launch_commit_t<16, bf16_bits>(a) : launch_commit_t<16, float>(a);
}

}  // namespace kda
