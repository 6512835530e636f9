// Norms around a block on gfx950 (kda.h: kda_gated_norm, kda_residual_norm).
//
// Both read every element once, keep a row in registers between the sum of its
// squares and its use, and write once: bound by HBM. A row belongs to L threads
// (4 to 64 lanes of a wave, then 128 to 1024 threads), each with up to I vectors
// of it, so that a wave holds several short rows and a long one fits. 8192 x 32 heads
// of 128, bf16: 37.5 us, 5.4 TB/s; residual norm of 8192 x 4096 with gate: 66 us, 5.1
// TB/s (a copy reaches 5.3 to 5.4).
#include "kda_pack.h"

namespace kda {
namespace {

// Sum over the L threads of a row (every one of them gets it). Rows of more than a
// wave: by way of LDS, in one of two places by turns (`turn`, the same for all), so
// that one barrier a sum is enough: a place is written again after the barrier of
// the sum between, which all of its readers have passed.
template <int L>
__device__ __forceinline__ float row_sum(float x, int& turn) {
  static_for<0, 6>([&](auto B) __attribute__((always_inline)) {
    constexpr int m = 1 << decltype(B)::value;
    if constexpr (m < L) x += lane_xor<m>(x);
  });
  if constexpr (L > kWave) {
    __shared__ float part[2][L / kWave];
    float* p = part[turn];
    turn ^= 1;
    if (threadIdx.x % kWave == 0) p[threadIdx.x / kWave] = x;
    lds_barrier();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < L / kWave; ++i) x += p[i];
  }
  return x;
}

// Most threads of a residual norm, whose workgroups then take several rows: four
// waves a SIMD. 4096 rows of 16384, bf16: 139 us, with two waves a SIMD 204, with
// eight 145, a workgroup for every row 180; 8192 of 4096: 65, 63, 69, 65.
constexpr int64_t kResidualThreads = 256 * 4 * 4 * 64;

// (a row of more than a wave has a workgroup to itself)
template <int L> constexpr int threads_of() { return L > kWave ? L : 256; }

// 1 / sqrt(mean of squares + eps) of a row whose threads hold v.
template <int L, int I, int V>
__device__ __forceinline__ float inv_rms(const float (&v)[I][V], int D, float eps, int& turn) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) s += v[i][e] * v[i][e];
  return rsqrtf(row_sum<L>(s, turn) * (1.0f / (float)D) + eps);
}

template <typename T, int V, bool whole, int L, int I>
__global__ __launch_bounds__(threads_of<L>()) void gated_norm_kernel(const T* x, int64_t x_stride, const T* gate,
                                                                     int64_t gate_stride, const float* weight,
                                                                     bool per_head, int64_t rows, int H, int D, int act,
                                                                     bool gate_first, float eps, T* y) {
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * (threads_of<L>() / L) + threadIdx.x / L;
  // (threads without a row stay for the sums of their wave)
  const bool live = r < rows;
  const int64_t t = live ? r / H : 0;
  const int h = live ? (int)(r % H) : 0;
  const T* px = x + t * x_stride + (int64_t)h * D;
  const T* pg = gate ? gate + t * gate_stride + (int64_t)h * D : nullptr;
  float v[I][V], g[I][V];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const VecAt<V, whole> at = vec_at<V, whole>(lane + i * L, D);
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = 0.f, g[i][e] = 1.f;
    if (live && at.on) {
      from_bits<T, V>(load_row<whole, T, V>(px + at.c, D), v[i]);
      if (at.skip) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = e < at.skip ? 0.f : v[i][e];
      }
      if (pg) {
        from_bits<T, V>(load_row<whole, T, V>(pg + at.c, D), g[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) g[i][e] = activate<T>(g[i][e], act);
      }
    }
    if (gate_first) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = e < at.skip ? 0.f : v[i][e] * g[i][e], g[i][e] = 1.f;
    }
  }
  int turn = 0;
  const float s = inv_rms<L, I, V>(v, D, eps, turn);
  if (!live) return;
  const float* w = weight + (per_head ? (int64_t)h * D : 0);
  T* py = y + r * D;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const VecAt<V, whole> at = vec_at<V, whole>(lane + i * L, D);
    if (at.on) {
      float o[V];
      load_params<V>(w + at.c, min(V, D), 0.f, o);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= v[i][e] * s * g[i][e];
      store_row<whole, T, V>(py + at.c, to_bits<T, V>(o), at.skip, D);
    }
  }
}

// A workgroup takes rows `step` apart, with its columns' weights in registers for
// all of them (they are fp32: a row's weights are more bytes than the row) and the
// next row's loads on their way while it works on one. Rows of more than 8192 elements
// leave no registers for the weights: they are read for each row.
template <typename T, int V, bool whole, int L, int I>
__global__ __launch_bounds__(threads_of<L>()) void residual_norm_kernel(const T* x, const T* residual, const T* gate,
                                                                        const float* weight, const float* post,
                                                                        const float* scale, int64_t rows, int64_t step,
                                                                        int C, int act, float alpha, float eps,
                                                                        T* residual_out, T* y) {
  const int lane = threadIdx.x % L;
  const int64_t r0 = (int64_t)blockIdx.x * (threads_of<L>() / L);
  constexpr bool kKeep = I * V < 16;
  float w[I][V], pw[I][V], k[I][V];
  bits_t<T, V> nx[I] = {}, nr[I] = {}, ng[I] = {};
  auto vec = [&](int i) { return vec_at<V, whole>(lane + i * L, C); };
  // (threads without a row stay for the sums of their wave)
  auto load = [&](int64_t r) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (r < rows && vec(i).on) {
        const int64_t at = r * C + vec(i).c;
        nx[i] = load_row<whole, T, V>(x + at, C);
        if (residual) nr[i] = load_row<whole, T, V>(residual + at, C);
        if (gate) ng[i] = load_row<whole, T, V>(gate + at, C);
      }
  };
  load(r0 + threadIdx.x / L);
  auto params = [&](int i) __attribute__((always_inline)) {
    const int c = vec(i).c;
#pragma unroll
    for (int e = 0; e < V; ++e) pw[i][e] = k[i][e] = 1.f;
    if (vec(i).on) {
      if (post) load_params<V>(post + c, min(V, C), 0.f, pw[i]);
      if (scale) load_params<V>(scale + c, min(V, C), 0.f, k[i]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) k[i][e] *= alpha;
  };
  auto weights = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[i][e] = 0.f;
    if (vec(i).on) load_params<V>(weight + vec(i).c, min(V, C), 0.f, w[i]);
  };
  if (kKeep)
#pragma unroll
    for (int i = 0; i < I; ++i) params(i), weights(i);
  const int64_t mine = threadIdx.x / L;
  int turn = 0;
  for (int64_t rb = r0; rb < rows; rb += step) {
    const int64_t r = rb + mine;
    float v[I][V], res[I][V], g[I][V];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      from_bits<T, V>(nx[i], v[i]);
      from_bits<T, V>(nr[i], res[i]);
      from_bits<T, V>(ng[i], g[i]);
      const int skip = vec(i).skip;
      if (skip) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] = e < skip ? 0.f : v[i][e];
      }
    }
    load(r + step);
    const float s = post ? inv_rms<L, I, V>(v, C, eps, turn) : 1.f;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const VecAt<V, whole> at = vec(i);
      if (!kKeep) params(i);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = v[i][e];
        if (post) u = u * s * pw[i][e];
        if (gate) u *= activate<T>(g[i][e], act);
        // (columns of the vector in front, and behind the row's last, count for nothing)
        v[i][e] = at.owns(e, C) ? res[i][e] + k[i][e] * u : 0.f;
      }
    }
    const bool live = r < rows;
    if (residual_out)
#pragma unroll
      for (int i = 0; i < I; ++i)
        if (live && vec(i).on) store_row<whole, T, V>(residual_out + r * C + vec(i).c, to_bits<T, V>(v[i]), vec(i).skip, C);
    const float q = inv_rms<L, I, V>(v, C, eps, turn);
#pragma unroll
    for (int i = 0; i < I; ++i)
      if (live && vec(i).on) {
        if (!kKeep) weights(i);
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = v[i][e] * q * w[i][e];
        store_row<whole, T, V>(y + r * C + vec(i).c, to_bits<T, V>(o), vec(i).skip, C);
      }
  }
}

// Calls f(integral L, integral I) with the fewest threads and vectors a thread
// that hold n vectors.
template <int V, typename F>
void by_length(int n, F&& f) {
#define KDA_ROW(l, i) f(std::integral_constant<int, l>{}, std::integral_constant<int, i>{})
  if (n <= 4) KDA_ROW(4, 1);
  else if (n <= 8) KDA_ROW(8, 1);
  else if (n <= 16) KDA_ROW(16, 1);
  else if (n <= 32) KDA_ROW(32, 1);
  else if (n <= 64) KDA_ROW(64, 1);
  else if (n <= 128) KDA_ROW(128, 1);
  else if (n <= 256) KDA_ROW(256, 1);
  else if (n <= 512) KDA_ROW(512, 1);
  else if (n <= 1024) KDA_ROW(1024, 1);
  else if (V > 4 || n <= 2048) KDA_ROW(1024, 2);
  else if constexpr (V <= 4) KDA_ROW(1024, 4);
#undef KDA_ROW
}
static_assert(KDA_NORM_MAX <= 1024 * 2 * 8 && KDA_NORM_MAX <= 1024 * 4 * 4, "longest rows");

template <typename T, int V, bool whole>
void gated_t(const GatedNormArgs& a) {
  const int64_t rows = (int64_t)a.T * a.H;
  by_length<V>((a.D + V - 1) / V, [&](auto L, auto I) {
    constexpr int l = decltype(L)::value, i = decltype(I)::value, per = threads_of<l>() / l;
    hipLaunchKernelGGL((gated_norm_kernel<T, V, whole, l, i>), dim3((unsigned)((rows + per - 1) / per)),
                       dim3(threads_of<l>()), 0, a.stream, (const T*)a.x, a.x_stride, (const T*)a.gate, a.gate_stride,
                       a.weight, a.weight_per_head, rows, a.H, a.D, a.act, a.gate_first, a.eps, (T*)a.y);
  });
}
template <typename T, int V, bool whole>
void residual_t(const ResidualNormArgs& a) {
  by_length<V>((a.C + V - 1) / V, [&](auto L, auto I) {
    constexpr int l = decltype(L)::value, i = decltype(I)::value, per = threads_of<l>() / l;
    int64_t groups = ((int64_t)a.T + per - 1) / per;
    const int64_t most = kResidualThreads / threads_of<l>();
    if (groups > most) groups = most;
    hipLaunchKernelGGL((residual_norm_kernel<T, V, whole, l, i>), dim3((unsigned)groups), dim3(threads_of<l>()), 0, a.stream,
                       (const T*)a.x, (const T*)a.residual, (const T*)a.gate, a.weight, a.post_weight, a.scale,
                       (int64_t)a.T, groups * per, a.C, a.act, a.alpha, a.eps, (T*)a.residual_out, (T*)a.y);
  });
}
template <int V>
int64_t row_threads(int64_t rows, int n) {
  int64_t t = 0;
  by_length<V>(n, [&](auto L, auto) { t = (rows + 255) * decltype(L)::value; });
  return t;
}

}  // namespace

int64_t gated_threads(const GatedNormArgs& a) {
  const int64_t rows = (int64_t)a.T * a.H;
  return a.bf16 ? row_threads<8>(rows, (a.D + 7) / 8) : row_threads<4>(rows, (a.D + 3) / 4);
}

hipError_t launch_gated_norm(const GatedNormArgs& a) {
  if (a.bf16) a.D % 8 == 0 ? gated_t<bf16_bits, 8, true>(a) : gated_t<bf16_bits, 8, false>(a);
  else a.D % 4 == 0 ? gated_t<float, 4, true>(a) : gated_t<float, 4, false>(a);
  return hipGetLastError();
}

hipError_t launch_residual_norm(const ResidualNormArgs& a) {
  if (a.bf16) a.C % 8 == 0 ? residual_t<bf16_bits, 8, true>(a) : residual_t<bf16_bits, 8, false>(a);
  else a.C % 4 == 0 ? residual_t<float, 4, true>(a) : residual_t<float, 4, false>(a);
  return hipGetLastError();
}

}  // namespace kda
