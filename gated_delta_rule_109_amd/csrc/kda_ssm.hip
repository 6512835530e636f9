// Selective state-space scan over packed sequences on gfx950, for prompts and
// for single tokens (kda.h: kda_ssm_prefill, kda_ssm_step).
//
//   S_t = exp(d_t a) S_{t-1} + d_t b_t x_t^T,   y_t = S_t^T c_t + skip x_t
//
// One decay per head and token; S is N x P in fp32.
#include "kda_pack.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 64;         // columns of a head one workgroup owns
constexpr int kGroupTarget = 1024;   // workgroups that segments of one sequence make up
constexpr int kMinSegment = 128;     // tokens

// Segments. A call with few sequences, heads and columns cuts its sequences
// every segment_len tokens, and the segments run side by side in two launches:
//   1: every segment but the last of its sequence, from a zero state, for its
//      last state alone; the first segment from the initial state and with its
//      outputs.
//   2: the segments behind the first, from the state in front of them,
//      S(j) = end_0 carried over segments 1 .. j - 1: S <- e^{sum d a} S + end_i.
// Nothing in the second launch reads initial states, so they may be the final
// ones. (segment j of a sequence that starts at token s stores its last state
// at entry s / len + j: sequences have fewer entries than segments, so no two
// meet.)
int segment_len(const Packed& s, int H, int P) {
  const int64_t groups = (int64_t)H * ((P + kColumns - 1) / kColumns);
  const int64_t parts = kGroupTarget / groups;          // segments all sequences have together
  if (parts < 2 || s.T < 2 * kMinSegment) return s.T > 0 ? s.T : 1;
  const int64_t len = ((s.T + parts - 1) / parts + KDA_SSM_CHUNK - 1) / KDA_SSM_CHUNK * KDA_SSM_CHUNK;
  return (int)(len > kMinSegment ? len : kMinSegment);
}

// d_t of one token and head.
__device__ __forceinline__ float step_size(float dt, float bias, bool softplus) {
  const float v = dt + bias;
  // ln(1 + e^v) = max(v, 0) + ln(1 + e^-|v|); NaN stays NaN
  return softplus ? (v > 0.f ? v : v < 0.f ? 0.f : v) + log1pf(expf(-fabsf(v))) : v;
}

struct SsmParams {
  const void *x, *b, *c;
  int64_t x_stride, b_stride, c_stride;
  const float *dt, *a, *skip, *dt_bias;
  bool softplus;
  Packed seqs;
  int H, G, P, len;
  const float* initial_state;
  float* final_state;
  void* y;
  float* ends;      // last states of segments [entry][H][P blocks][..]
  double* sums;     // sum of d a over them [entry][H]
};

// Token by token in fp32. A workgroup owns kColumns columns of one head: wave w
// the 16 columns 16 w .., lane l column l % 16 and the N / 4 rows
// 16 i + 4 (l / 16) + 0..3. Tokens are staged kStage at a time.
constexpr int kStage = 16;

template <typename T, int N>
__global__ __launch_bounds__(kThreads) void ssm_token_kernel(SsmParams a, int pass) {
  const int pblocks = (a.P + kColumns - 1) / kColumns;
  const int pb = blockIdx.x % pblocks, h = blockIdx.x / pblocks % a.H;
  Part p;
  if (!find_part(a.seqs, a.len, blockIdx.x / pblocks / a.H, p)) return;
  const bool last = p.j == p.parts - 1;
  if (pass == 1 ? last && p.j > 0 : p.j == 0) return;
  const bool outputs = pass == 2 || p.j == 0;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, q = lane / 16;
  const int col = pb * kColumns + wave * 16 + lane % 16;
  const bool live = pb * kColumns + wave * 16 < a.P;    // (P is a multiple of 16)
  const int grp = h / (a.H / a.G);
  constexpr int R = N / 16;
  f32x4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const size_t state = ((size_t)p.n * a.H + h) * N * a.P + col;
  auto entry = [&](int j) { return ((size_t)(p.start / a.len + j) * a.H + h); };
  auto end_of = [&](int j) { return (f32x4*)a.ends + (entry(j) * pblocks + pb) * (R * kThreads) + tid; };
  if (live) {
    if (p.j == 0) {
      if (a.initial_state)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = a.initial_state[state + (size_t)(16 * i + 4 * q + e) * a.P];
    } else if (pass == 2) {
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = end_of(0)[i * kThreads];
      for (int j = 1; j < p.j; ++j) {
        const float f = __builtin_amdgcn_exp2f((float)(a.sums[entry(j)] * 1.4426950408889634));
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = f * s[i] + end_of(j)[i * kThreads];
      }
    }
  }
  __shared__ float sb[kStage][N], sc[kStage][N], sx[kStage][kColumns], sf[kStage], sd[kStage];
  const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.skip ? a.skip[h] : 0.f;
  double sum = 0.0;
  for (int t0 = 0; t0 < p.count; t0 += kStage) {
    const int m = min(kStage, p.count - t0);
    const int64_t tok = p.first + t0;
    __syncthreads();
    for (int e = tid; e < m * N; e += kThreads) {
      const int t = e / N, i = e % N;
      sb[t][i] = Elem<T>::load((const T*)a.b + (tok + t) * a.b_stride + grp * N + i);
      sc[t][i] = Elem<T>::load((const T*)a.c + (tok + t) * a.c_stride + grp * N + i);
    }
    for (int e = tid; e < m * kColumns; e += kThreads) {
      const int t = e / kColumns, i = pb * kColumns + e % kColumns;
      if (i < a.P) sx[t][e % kColumns] = Elem<T>::load((const T*)a.x + (tok + t) * a.x_stride + (int64_t)h * a.P + i);
    }
    if (tid < m) {
      const float d = step_size(a.dt[(tok + tid) * a.H + h], bias, a.softplus);
      sd[tid] = d;
      sf[tid] = expf(d * av);
      sum += (double)d * av;
    }
    __syncthreads();
    if (live) {
      for (int t = 0; t < m; ++t) {
        const float xv = sx[t][wave * 16 + lane % 16], f = sf[t], dx = sd[t] * xv;
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const f32x4 b = *(const f32x4*)&sb[t][16 * i + 4 * q], c = *(const f32x4*)&sc[t][16 * i + 4 * q];
          s[i] = f * s[i] + b * dx;
#pragma unroll
          for (int e = 0; e < 4; ++e) o += s[i][e] * c[e];
        }
        if (outputs) {
          o += lane_xor<16>(o);
          o += lane_xor<32>(o);
          if (q == 0) Elem<T>::store((T*)a.y + ((size_t)(tok + t) * a.H + h) * a.P + col, a.skip ? o + skip * xv : o);
        }
      }
    }
  }
  if (!last) {
    if (live)
#pragma unroll
      for (int i = 0; i < R; ++i) end_of(p.j)[i * kThreads] = s[i];
    if (p.j > 0 && pb == 0 && wave == 0) {
      for (int m = 1; m < kStage; m *= 2) sum += __shfl_xor(sum, m);
      if (tid == 0) a.sums[entry(p.j)] = sum;
    }
  } else if (a.final_state && live) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) a.final_state[state + (size_t)(16 * i + 4 * q + e) * a.P] = s[i][e];
  }
}

// One token: the state read and written once, a float4 of columns per thread
// and 256 / (P / 4) rows at a time (the rest of the workgroup idles where P / 4
// does not divide it).
template <typename T>
__global__ __launch_bounds__(kThreads) void ssm_step_kernel(SsmParams a, int N) {
  const int h = blockIdx.x % a.H, n = blockIdx.x / a.H;
  const int vecs = a.P / 4, groups = kThreads / vecs;
  const int tid = threadIdx.x, cv = tid % vecs, rg = tid / vecs;
  const int grp = h / (a.H / a.G);
  __shared__ float sb[256], sc[256];
  __shared__ f32x4 part[kThreads];
  const float d = step_size(a.dt[(size_t)n * a.H + h], a.dt_bias ? a.dt_bias[h] : 0.f, a.softplus);
  const float f = expf(d * a.a[h]);
  if (tid < N) {
    sb[tid] = d * Elem<T>::load((const T*)a.b + n * a.b_stride + grp * N + tid);
    sc[tid] = Elem<T>::load((const T*)a.c + n * a.c_stride + grp * N + tid);
  }
  __syncthreads();
  float xv[4];
  load_vec<T, 4>((const T*)a.x + n * a.x_stride + (int64_t)h * a.P + cv * 4, xv);
  const f32x4 x = {xv[0], xv[1], xv[2], xv[3]};
  float* S = a.final_state + ((size_t)n * a.H + h) * N * a.P + cv * 4;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  if (rg < groups) {
    constexpr int U = 4;
    for (int r0 = rg; r0 < N; r0 += U * groups) {
      f32x4 s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = *(const f32x4*)(S + (size_t)min(r0 + u * groups, N - 1) * a.P);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * groups;
        if (r < N) {
          s[u] = f * s[u] + sb[r] * x;
          o += sc[r] * s[u];
          *(f32x4*)(S + (size_t)r * a.P) = s[u];
        }
      }
    }
    part[tid] = o;
  }
  __syncthreads();
  if (tid < vecs) {
    for (int g = 1; g < groups; ++g) o += part[g * vecs + tid];
    if (a.skip) o += a.skip[h] * x;
    const float out[4] = {o[0], o[1], o[2], o[3]};
    store_vec<T, 4>((T*)a.y + ((size_t)n * a.H + h) * a.P + cv * 4, out);
  }
}

SsmParams params_of(const SsmArgs& a, int len) {
  SsmParams p;
  p.x = a.x; p.b = a.b; p.c = a.c;
  p.x_stride = a.x_stride; p.b_stride = a.b_stride; p.c_stride = a.c_stride;
  p.dt = a.dt; p.a = a.a; p.skip = a.skip; p.dt_bias = a.dt_bias;
  p.softplus = a.softplus;
  p.seqs = a.seqs;
  p.H = a.H; p.G = a.G; p.P = a.P; p.len = len;
  p.initial_state = a.initial_state; p.final_state = a.final_state;
  p.y = a.y;
  p.ends = nullptr; p.sums = nullptr;
  return p;
}

int64_t entries(const Packed& s, int len) { return len < s.T ? s.T / len : 0; }
size_t end_bytes(int H, int N, int P) { return (size_t)H * ((P + kColumns - 1) / kColumns) * kColumns * N * 4; }

template <typename T, int N>
hipError_t launch_n(const SsmArgs& a) {
  const int len = segment_len(a.seqs, a.H, a.P);
  SsmParams p = params_of(a, len);
  const int64_t e = entries(a.seqs, len);
  p.ends = (float*)a.workspace;
  p.sums = (double*)((char*)a.workspace + e * end_bytes(a.H, N, a.P));
  const unsigned groups = (unsigned)ssm_groups(a);
  for (int pass = 1; pass <= (e > 0 ? 2 : 1); ++pass)
    hipLaunchKernelGGL((ssm_token_kernel<T, N>), dim3(groups), dim3(kThreads), 0, a.stream, p, pass);
  return hipGetLastError();
}
template <typename T>
hipError_t launch_t(const SsmArgs& a) {
  switch (a.N) {
    case 16: return launch_n<T, 16>(a);
    case 32: return launch_n<T, 32>(a);
    case 64: return launch_n<T, 64>(a);
    case 128: return launch_n<T, 128>(a);
    default: return launch_n<T, 256>(a);
  }
}

}  // namespace

int64_t ssm_groups(const SsmArgs& a) {
  return part_slots(a.seqs, segment_len(a.seqs, a.H, a.P)) * a.H * ((a.P + kColumns - 1) / kColumns);
}

// At most kGroupTarget / groups segments of one sequence's worth, and at most
// one per kMinSegment tokens: both grow with the sizes.
size_t ssm_workspace(int32_t num_seqs, int32_t T, int32_t H, int32_t N, int32_t P) {
  (void)num_seqs;
  const size_t by_target = (size_t)kGroupTarget * kColumns * N * 4 + (size_t)kGroupTarget * 8;
  const size_t by_length = (size_t)(T / kMinSegment) * (end_bytes(H, N, P) + (size_t)H * 8);
  return by_target < by_length ? by_target : by_length;
}

hipError_t launch_ssm(const SsmArgs& a) { return a.bf16 ? launch_t<bf16_bits>(a) : launch_t<float>(a); }

hipError_t launch_ssm_step(const SsmArgs& a) {
  SsmParams p = params_of(a, 1);
  const dim3 grid((unsigned)((int64_t)a.seqs.num_seqs * a.H));
  if (a.bf16) hipLaunchKernelGGL(ssm_step_kernel<bf16_bits>, grid, dim3(kThreads), 0, a.stream, p, a.N);
  else hipLaunchKernelGGL(ssm_step_kernel<float>, grid, dim3(kThreads), 0, a.stream, p, a.N);
  return hipGetLastError();
}

}  // namespace kda
