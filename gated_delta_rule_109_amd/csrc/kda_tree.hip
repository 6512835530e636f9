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

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float x) {
  x += lane_xor<1>(x); x += lane_xor<2>(x); x += lane_xor<4>(x);
  x += lane_xor<8>(x); x += lane_xor<16>(x); x += lane_xor<32>(x);
  return x;
}

// Decay of one channel of token row `row` (a row of the [N, T, H] grid).
__device__ __forceinline__ float load_alpha(const float* g, int gate, size_t row, int D, int c, uint32_t fe_flags,
                                            float g_min, float alpha_min) {
  if (gate == KDA_GATE_NONE) return 1.f;
  const float x = g[gate == KDA_GATE_CHANNEL ? row * D + c : row];
  return fe_flags & KDA_FE_GATE_LOGITS ? gate_alpha_logit(x, alpha_min) : gate_alpha(x, g_min);
}

// The parent of node i as the kernels use it: -1 unless in [0, i - 1].
__device__ __forceinline__ int clean_parent(const int32_t* parents, size_t first, int i) {
  if (!parents) return i - 1;
  const int p = parents[first + i];
  return p >= 0 && p < i ? p : -1;
}

// ---- any decays, any head size -------------------------------------------------
// One 256-thread workgroup per (sequence, head). A_ij and B_ij are summed pair
// by pair along each node's path, with the decay between the two nodes built
// up factor by factor on the way to the root, so no quotient of decays is ever
// formed and any floor works; only a node's own ancestors are touched.
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
    int T, float scale, float g_min, uint32_t fe_flags, float fe_eps, int gate) {
  const uint32_t n = blockIdx.x / (uint32_t)H, h = blockIdx.x % (uint32_t)H;
  const int nt = num_nodes ? min(max(num_nodes[n], 0), T) : T;
  if (nt == 0) return;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
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

template <int D, typename TIn>
static hipError_t launch_tree_t(const TreeArgs& a) {
  const unsigned blocks = (unsigned)((int64_t)a.N * a.H);
  hipLaunchKernelGGL((tree_path_kernel<D, TIn>), dim3(blocks), dim3(256), path_lds_bytes<D>(a.T), a.stream,
                     (const TIn*)a.q, (const TIn*)a.k, (const TIn*)a.v, a.g, a.beta, a.state, a.parents,
                     a.num_nodes, (TIn*)a.o, a.H, a.T, a.scale, a.g_min, a.fe_flags, a.fe_eps, (int)a.gate);
  return hipGetLastError();
}

hipError_t launch_tree(const TreeArgs& a) {
  if (a.D == 128) return a.bf16 ? launch_tree_t<128, bf16_bits>(a) : launch_tree_t<128, float>(a);
  return a.bf16 ? launch_tree_t<16, bf16_bits>(a) : launch_tree_t<16, float>(a);
}

// ---- commit of a path -------------------------------------------------------------
// The recurrence over the accepted nodes, the state in registers from its one
// read to its one write (8 D^2 bytes per head, which is what the call costs).
// Thread layout as the decode kernel's: D = 128, a 256-thread workgroup per
// head, lane l of wave w owns columns 32w + 4(l % 8) .. +3 of rows
// (l / 8) + 8i; D = 16, one wave per head.
// The nodes' vectors are staged kBatch nodes at a time; the first batch is
// loaded ahead of the state so that both are in flight together.
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
  // the path's length: accept, cut before the first index outside [0, T)
  const int node_of_lane = path[(size_t)n * T + min(lane, T - 1)];
  const uint64_t bad = __ballot(!(lane < T && node_of_lane >= 0 && node_of_lane < T));
  int len = min(max(accept[n], 0), T);
  if (bad) len = min(len, __builtin_ctzll(bad));
  if (len == 0) return;
  const int cg = lane % kColGroups, rg = lane / kColGroups;
  const int col = wave * 4 * kColGroups + 4 * cg;
  auto row = [&](int i) __attribute__((always_inline)) {
    return ((size_t)n * T + path[(size_t)n * T + i]) * H + h;
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
    if (tid < kBatch) tb = beta[row(min(first + tid, len - 1))];
  };
  auto stage = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int x = 0; x < kIters; ++x) {
      const int e = tid + x * kThreads, t = e / D, c = e % D;
      s_k[t][c] = tk[x];
      s_v[t][c] = tv[x];
      s_a[t][c] = gate == KDA_GATE_NONE              ? 1.f
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
