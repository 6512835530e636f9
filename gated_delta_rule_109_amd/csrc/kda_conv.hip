// Short causal convolution over packed sequences on gfx950, for prompts and for
// single tokens (kda.h: kda_conv_prefill, kda_conv_step).
//
//   y[t][c] = act(bias[c] + sum_j w[c][j] x[t - K + 1 + j][c])
//
// 2 K operations and the activation per element against 2 elements of traffic:
// bound by HBM. A thread owns V consecutive channels (16 bytes) and walks along
// the tokens with the last K - 1 rows in registers, so every row is read once
// but for the K - 1 rows in front of a thread's first token.
#include "kda_pack.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 32;   // tokens a thread walks along

// Threads along the channels; the rest of the workgroup takes further tokens.
int channel_threads(int vecs) {
  int t = 1;
  while (t < vecs && t < kThreads) t *= 2;
  return t;
}

template <typename T, int V, int K>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int c, float (&w)[V][K],
                                             float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[i][j] = weight[(size_t)(c + i) * K + j];
    b[i] = bias ? bias[c + i] : 0.f;
  }
}

// Output of one token from its row and the K - 1 rows before it; shifts the rows.
template <typename T, int V, int K>
__device__ __forceinline__ void conv_token(float (&past)[K - 1][V], const float (&x)[V], const float (&w)[V][K],
                                           const float (&b)[V], bool silu, T* y) {
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = b[i];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) s += w[i][j] * past[j][i];
    s += w[i][K - 1] * x[i];
    out[i] = silu ? s * sigmoid<T>(s) : s;
#pragma unroll
    for (int j = 0; j < K - 2; ++j) past[j][i] = past[j + 1][i];
    past[K - 2][i] = x[i];
  }
  store_vec<T, V>(y, out);
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_kernel(const T* x, int64_t x_stride, const float* weight,
                                                        const float* bias, Packed seqs, int C, int chan_threads,
                                                        int chan_blocks, bool silu, const T* initial, T* final_state,
                                                        T* y) {
  const int cb = blockIdx.x % chan_blocks, slot = blockIdx.x / chan_blocks;
  const int c = (cb * chan_threads + (int)threadIdx.x % chan_threads) * V;
  const int row = threadIdx.x / chan_threads;     // which run of kTokens tokens
  Part p;
  if (!find_part(seqs, kThreads / chan_threads * kTokens, slot, p) || c >= C) return;
  const int first = p.first + row * kTokens;
  const int count = min(kTokens, p.first + p.count - first);
  // the rows in front: of the sequence, or of its state (row r of the state is
  // token start - (K - 1) + r)
  float past[K - 1][V] = {};
  if (count > 0) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = first - (K - 1) + j;
      if (t >= p.start) load_vec<T, V>(x + t * x_stride + c, past[j]);
      else if (initial) load_vec<T, V>(initial + ((size_t)p.n * (K - 1) + t - p.start + K - 1) * C + c, past[j]);
    }
    float w[V][K], b[V];
    load_weights<T, V, K>(weight, bias, c, w, b);
    constexpr int U = 4;   // rows in flight
    for (int t0 = 0; t0 < count; t0 += U) {
      float rows[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        load_vec<T, V>(x + (int64_t)(first + min(t0 + u, count - 1)) * x_stride + c, rows[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + u < count) conv_token<T, V, K>(past, rows[u], w, b, silu, y + (size_t)(first + t0 + u) * C + c);
    }
  }
  // The state after the sequence, by the threads that alone read the state
  // before it (the first K - 1 tokens are theirs): it may be the same array.
  // Row i comes from row length + i of the state, not from a row before i.
  if (final_state && p.j == 0 && row == 0) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int t = p.length - (K - 1) + i;
      Pack<T, V> v = {};
      if (t >= 0) v = *(const Pack<T, V>*)(x + (int64_t)(p.start + t) * x_stride + c);
      else if (initial) v = *(const Pack<T, V>*)(initial + ((size_t)p.n * (K - 1) + p.length + i) * C + c);
      *(Pack<T, V>*)(final_state + ((size_t)p.n * (K - 1) + i) * C + c) = v;
    }
  }
}
static_assert(kTokens >= KDA_CONV_MAX_WIDTH - 1, "the first K - 1 tokens are one thread's");

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(const T* x, int64_t x_stride, const float* weight,
                                                             const float* bias, int N, int C, bool silu, T* state,
                                                             T* y) {
  const int vecs = C / V;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (id >= (int64_t)N * vecs) return;
  const int n = id / vecs, c = (int)(id % vecs) * V;
  T* s = state + (size_t)n * (K - 1) * C + c;
  float past[K - 1][V], in[V], w[V][K], b[V];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) load_vec<T, V>(s + (size_t)j * C, past[j]);
  load_vec<T, V>(x + n * x_stride + c, in);
  load_weights<T, V, K>(weight, bias, c, w, b);
  conv_token<T, V, K>(past, in, w, b, silu, y + (size_t)n * C + c);
#pragma unroll
  for (int j = 0; j < K - 1; ++j) store_vec<T, V>(s + (size_t)j * C, past[j]);
}

// Whether rows of C elements at these strides are vectors of V elements.
template <typename T, int V>
bool vectors(const ConvArgs& a) {
  return a.C % V == 0 && a.x_stride % V == 0;
}

template <typename T, int V, int K>
hipError_t conv_t(const ConvArgs& a) {
  const int ct = channel_threads(a.C / V), blocks = (a.C / V + ct - 1) / ct;
  const int64_t slots = part_slots(a.seqs, kThreads / ct * kTokens);
  hipLaunchKernelGGL((conv_kernel<T, V, K>), dim3((unsigned)(slots * blocks)), dim3(kThreads), 0, a.stream,
                     (const T*)a.x, a.x_stride, a.weight, a.bias, a.seqs, a.C, ct, blocks, a.silu,
                     (const T*)a.initial_state, (T*)a.final_state, (T*)a.y);
  return hipGetLastError();
}
template <typename T, int V, int K>
hipError_t step_t(const ConvArgs& a) {
  const int64_t n = (int64_t)a.N * (a.C / V);
  hipLaunchKernelGGL((conv_step_kernel<T, V, K>), dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                     a.stream, (const T*)a.x, a.x_stride, a.weight, a.bias, a.N, a.C, a.silu, (T*)a.initial_state,
                     (T*)a.y);
  return hipGetLastError();
}

template <typename T, int V>
hipError_t by_width(const ConvArgs& a, bool step) {
  switch (a.width) {
    case 2: return step ? step_t<T, V, 2>(a) : conv_t<T, V, 2>(a);
    case 3: return step ? step_t<T, V, 3>(a) : conv_t<T, V, 3>(a);
    default: return step ? step_t<T, V, 4>(a) : conv_t<T, V, 4>(a);
  }
}
hipError_t by_type(const ConvArgs& a, bool step) {
  if (a.bf16) return vectors<bf16_bits, 8>(a) ? by_width<bf16_bits, 8>(a, step) : by_width<bf16_bits, 1>(a, step);
  return vectors<float, 4>(a) ? by_width<float, 4>(a, step) : by_width<float, 1>(a, step);
}

}  // namespace

int64_t conv_threads(const ConvArgs& a, bool step) {
  const int v = a.bf16 ? (vectors<bf16_bits, 8>(a) ? 8 : 1) : (vectors<float, 4>(a) ? 4 : 1);
  if (step) return (int64_t)a.N * (a.C / v) + kThreads;
  const int ct = channel_threads(a.C / v);
  return part_slots(a.seqs, kThreads / ct * kTokens) * ((a.C / v + ct - 1) / ct) * kThreads;
}

hipError_t launch_conv(const ConvArgs& a) { return by_type(a, false); }
hipError_t launch_conv_step(const ConvArgs& a) { return by_type(a, true); }

}  // namespace kda
