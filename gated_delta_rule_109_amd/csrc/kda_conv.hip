// Short causal convolution over packed sequences on gfx950, for prompts and for
// single tokens (kda.h: kda_conv_prefill, kda_conv_step).
//
//   y[t][c] = act(bias[c] + sum_j w[c][j] x[t - K + 1 + j][c])
//
// 2 K operations and the activation per element against 2 elements of traffic:
// bound by HBM. A thread owns V consecutive channels (16 bytes, or what a row has
// left) and walks along the tokens with the last K - 1 rows in registers, so every
// row is read once but for the K - 1 rows in front of a thread's first token; four
// rows are on their way while four are worked on. 8192 x 12288 bf16: 88 us, 4.6 TB/s,
// where a copy of the same bytes takes 75 (without the activation the same: it is not
// arithmetic); nine sequences of 3001 x 777 fp32 8.8 us one call after another, 10 alone.
#include "kda_pack.h"

namespace kda {
namespace {

// A workgroup is a wave: nothing in it waits for another one (prompts of 8192 x 12288
// bf16 88 us, by four waves 90; 24576 x 4096 81 and 85; 1 x 12288 3.5 and 4.4; steps of
// 256 x 12288 10.0 and 10.3, of 64 4.1 and 4.6).
constexpr int kGroup = kWave;
// Tokens a thread walks along: as many as leave kPromptThreads threads (two waves a
// SIMD), so that the rows in front of them are read seldom, and at least the K - 1
// that read the state. 2048 tokens of 12288 channels, bf16: 22.9 us, with a wave a
// SIMD 25.4, with four 25.3; 8192 tokens by 8 a thread 105, by 16 96, by 64 89 (all by
// workgroups of four waves).
constexpr int kMinTokens = 4, kMostTokens = 64;
constexpr int64_t kPromptThreads = 256 * 4 * 2 * 64;

// Threads along the channels; the rest of the workgroup takes further tokens.
int channel_threads(int vecs) {
  int t = 1;
  while (t < vecs && t < kGroup) t *= 2;
  return t;
}

template <typename T> constexpr int vec_of() { return 16 / sizeof(T); }
int vecs_of(const ConvArgs& a) {
  const int v = a.bf16 ? vec_of<bf16_bits>() : vec_of<float>();
  return (a.C + v - 1) / v;
}

int tokens_of(const ConvArgs& a) {
  int t = kMinTokens;
  while (t < kMostTokens && (int64_t)a.seqs.T * vecs_of(a) / (2 * t) >= kPromptThreads) t *= 2;
  return t;
}

// Weights and bias of channels c .. c + n - 1.
template <int V, int K>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int c, int n, float (&w)[V * K],
                                             float (&b)[V]) {
  load_params<V * K>(weight + (size_t)c * K, n * K, 0.f, w);
  if (bias) load_params<V>(bias + c, n, 0.f, b);
  else
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
}

// Output of one token from its row and the K - 1 rows before it; shifts the rows.
template <typename T, int V, int K>
__device__ __forceinline__ bits_t<T, V> conv_token(float (&past)[K - 1][V], bits_t<T, V> row, const float (&w)[V * K],
                                                   const float (&b)[V], bool silu) {
  float x[V], out[V];
  from_bits<T, V>(row, x);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = b[i];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) s += w[i * K + j] * past[j][i];
    s += w[i * K + K - 1] * x[i];
    out[i] = silu ? s * sigmoid<T>(s) : s;
#pragma unroll
    for (int j = 0; j < K - 2; ++j) past[j][i] = past[j + 1][i];
    past[K - 2][i] = x[i];
  }
  return to_bits<T, V>(out);
}

template <typename T, int K, bool whole>
__global__ __launch_bounds__(kGroup) void conv_kernel(const T* x, int64_t x_stride, const float* weight,
                                                        const float* bias, Packed seqs, int C, int tokens,
                                                        int chan_threads, int chan_blocks, bool silu, const T* initial, T* final_state,
                                                        T* y) {
  constexpr int V = vec_of<T>();
  const int cb = blockIdx.x % chan_blocks, slot = blockIdx.x / chan_blocks;
  const VecAt<V, whole> at = vec_at<V, whole>(cb * chan_threads + (int)threadIdx.x % chan_threads, C);
  const int c = at.c;
  const int row = threadIdx.x / chan_threads;     // which run of `tokens` tokens
  Part p;
  if (!find_part(seqs, kGroup / chan_threads * tokens, slot, p) || !at.on) return;
  const int first = p.first + row * tokens;
  const int count = min(tokens, p.first + p.count - first);
  // the rows in front: of the sequence, or of its state (row r of the state is
  // token start - (K - 1) + r)
  float past[K - 1][V] = {};
  if (count > 0) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = first - (K - 1) + j;
      if (t >= p.start) from_bits<T, V>(load_row<whole, T, V>(x + t * x_stride + c, C), past[j]);
      else if (initial)
        from_bits<T, V>(load_row<whole, T, V>(initial + ((size_t)p.n * (K - 1) + t - p.start + K - 1) * C + c, C), past[j]);
    }
    float w[V * K], b[V];
    load_weights<V, K>(weight, bias, c, min(V, C), w, b);
    constexpr int U = 4;   // rows on their way while as many are worked on
    bits_t<T, V> rows[U], next[U];
    auto load = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        next[u] = load_row<whole, T, V>(x + (int64_t)(first + min(t0 + u, count - 1)) * x_stride + c, C);
    };
    load(0);
    for (int t0 = 0; t0 < count; t0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) rows[u] = next[u];
      if (t0 + U < count) load(t0 + U);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (t0 + u < count)
          store_row<whole, T, V>(y + (size_t)(first + t0 + u) * C + c, conv_token<T, V, K>(past, rows[u], w, b, silu), at.skip, C);
    }
  }
  // The state after the sequence, by the threads that alone read the state
  // before it (the first K - 1 tokens are theirs): it may be the same array. (A row's
  // last vector also reads channels of the one in front, maybe after they are written;
  // it writes nothing of them.)
  // Row i comes from row length + i of the state, not from a row before i.
  if (final_state && p.j == 0 && row == 0) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int t = p.length - (K - 1) + i;
      bits_t<T, V> v = {};
      if (t >= 0) v = load_row<whole, T, V>(x + (int64_t)(p.start + t) * x_stride + c, C);
      else if (initial) v = load_row<whole, T, V>(initial + ((size_t)p.n * (K - 1) + p.length + i) * C + c, C);
      store_row<whole, T, V>(final_state + ((size_t)p.n * (K - 1) + i) * C + c, v, at.skip, C);
    }
  }
}
static_assert(kMinTokens >= KDA_CONV_MAX_WIDTH - 1, "the first K - 1 tokens are one thread's");

// One token: a thread takes the sequences n, n + groups, .. for its channels, whose
// weights (more bytes than a row and its state) it reads once.
template <typename T, int K, bool whole>
__global__ __launch_bounds__(kGroup) void conv_step_kernel(const T* x, int64_t x_stride, const float* weight,
                                                             const float* bias, int N, int C, int vecs, int groups,
                                                             bool silu, T* state, T* y) {
  constexpr int V = vec_of<T>();
  const uint32_t id = blockIdx.x * kGroup + threadIdx.x;
  if (id >= (uint32_t)groups * vecs) return;
  const VecAt<V, whole> at = vec_at<V, whole>(id % vecs, C);
  const int c = at.c;
  float w[V * K], b[V];
  load_weights<V, K>(weight, bias, c, min(V, C), w, b);
  for (int n = id / vecs; n < N; n += groups) {
    T* s = state + (size_t)n * (K - 1) * C + c;
    bits_t<T, V> rows[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) rows[j] = load_row<whole, T, V>(s + (size_t)j * C, C);
    rows[K - 1] = load_row<whole, T, V>(x + n * x_stride + c, C);
    float past[K - 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) from_bits<T, V>(rows[j], past[j]);
    store_row<whole, T, V>(y + (size_t)n * C + c, conv_token<T, V, K>(past, rows[K - 1], w, b, silu), at.skip, C);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) store_row<whole, T, V>(s + (size_t)j * C, rows[j + 1], at.skip, C);
  }
}

// Sequences apart that a thread of a step takes: about kStepThreads threads, a wave a
// SIMD. 256 sequences of 12288 channels, bf16: 10.0 us, 5.0 TB/s; before whole vectors
// had a kernel of their own 10.9, with twice the threads 11.4, half of them 14.8, a
// thread for every sequence 15.1.
constexpr int64_t kStepThreads = 256 * 4 * 64;
int step_groups(const ConvArgs& a) {
  const int64_t g = kStepThreads / vecs_of(a);
  return (int)(g < 1 ? 1 : g < a.N ? g : a.N);
}

template <typename T, int K, bool whole>
hipError_t launch_k(const ConvArgs& a, bool step) {
  const int vecs = vecs_of(a);
  if (step) {
    const int groups = step_groups(a);
    const int64_t n = (int64_t)groups * vecs;
    hipLaunchKernelGGL((conv_step_kernel<T, K, whole>), dim3((unsigned)((n + kGroup - 1) / kGroup)), dim3(kGroup), 0,
                       a.stream, (const T*)a.x, a.x_stride, a.weight, a.bias, a.N, a.C, vecs, groups, a.silu,
                       (T*)a.initial_state, (T*)a.y);
    return hipGetLastError();
  }
  const int tokens = tokens_of(a), ct = channel_threads(vecs), blocks = (vecs + ct - 1) / ct;
  const int64_t slots = part_slots(a.seqs, kGroup / ct * tokens);
  hipLaunchKernelGGL((conv_kernel<T, K, whole>), dim3((unsigned)(slots * blocks)), dim3(kGroup), 0, a.stream, (const T*)a.x,
                     a.x_stride, a.weight, a.bias, a.seqs, a.C, tokens, ct, blocks, a.silu, (const T*)a.initial_state,
                     (T*)a.final_state, (T*)a.y);
  return hipGetLastError();
}
template <typename T, bool whole>
hipError_t launch_w(const ConvArgs& a, bool step) {
  switch (a.width) {
    case 2: return launch_k<T, 2, whole>(a, step);
    case 3: return launch_k<T, 3, whole>(a, step);
    default: return launch_k<T, 4, whole>(a, step);
  }
}
template <typename T>
hipError_t launch_t(const ConvArgs& a, bool step) {
  return a.C % vec_of<T>() == 0 ? launch_w<T, true>(a, step) : launch_w<T, false>(a, step);
}

}  // namespace

int64_t conv_groups(const ConvArgs& a) {
  const int vecs = vecs_of(a), ct = channel_threads(vecs);
  return part_slots(a.seqs, kGroup / ct * tokens_of(a)) * ((vecs + ct - 1) / ct);
}

hipError_t launch_conv(const ConvArgs& a) { return a.bf16 ? launch_t<bf16_bits>(a, false) : launch_t<float>(a, false); }
hipError_t launch_conv_step(const ConvArgs& a) {
  return a.bf16 ? launch_t<bf16_bits>(a, true) : launch_t<float>(a, true);
}

}  // namespace kda
