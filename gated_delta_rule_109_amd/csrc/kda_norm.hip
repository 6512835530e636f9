// Norms around a block on gfx950 (kda.h: kda_gated_norm, kda_residual_norm).
//
// Both read every element once, keep a row in registers between the sum of its
// squares and its use, and write once: bound by HBM. A row belongs to L threads
// (4 to 64 lanes of a wave, then 256 or 1024 threads), each with up to I vectors
// of it, so that a wave holds several short rows and a long one fits.
#include "kda_pack.h"

namespace kda {
namespace {

// Sum over the L threads of a row (every one of them gets it).
template <int L>
__device__ __forceinline__ float row_sum(float x) {
  static_for<0, 6>([&](auto B) __attribute__((always_inline)) {
    constexpr int m = 1 << decltype(B)::value;
    if constexpr (m < L) x += lane_xor<m>(x);
  });
  if constexpr (L > kWave) {
    __shared__ float part[L / kWave];
    __syncthreads();   // (an earlier sum's readers are done)
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < L / kWave; ++i) x += part[i];
  }
  return x;
}

template <int L> constexpr int threads_of() { return L > 256 ? L : 256; }

// 1 / sqrt(mean of squares + eps) of a row whose threads hold v.
template <int L, int I, int V>
__device__ __forceinline__ float inv_rms(const float (&v)[I][V], int D, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) s += v[i][e] * v[i][e];
  return 1.0f / sqrtf(row_sum<L>(s) / (float)D + eps);
}

template <typename T, int V, int L, int I>
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
    const int d = (lane + i * L) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = 0.f, g[i][e] = 1.f;
    if (live && d < D) {
      load_vec<T, V>(px + d, v[i]);
      if (pg) {
        load_vec<T, V>(pg + d, g[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) g[i][e] = activate<T>(g[i][e], act);
      }
    }
    if (gate_first) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= g[i][e], g[i][e] = 1.f;
    }
  }
  const float s = inv_rms<L, I, V>(v, D, eps);
  if (!live) return;
  const float* w = weight + (per_head ? (int64_t)h * D : 0);
  T* py = y + r * D;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int d = (lane + i * L) * V;
    if (d < D) {
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = v[i][e] * s * w[d + e] * g[i][e];
      store_vec<T, V>(py + d, o);
    }
  }
}

template <typename T, int V, int L, int I>
__global__ __launch_bounds__(threads_of<L>()) void residual_norm_kernel(const T* x, const T* residual, const T* gate,
                                                                        const float* weight, const float* post,
                                                                        const float* scale, int64_t rows, int C,
                                                                        int act, float alpha, float eps,
                                                                        T* residual_out, T* y) {
  const int lane = threadIdx.x % L;
  const int64_t r = (int64_t)blockIdx.x * (threads_of<L>() / L) + threadIdx.x / L;
  const bool live = r < rows;
  const int64_t base = live ? r * C : 0;
  float v[I][V], res[I][V];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * L) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = 0.f, res[i][e] = 0.f;
    if (live && c < C) {
      load_vec<T, V>(x + base + c, v[i]);
      if (residual) load_vec<T, V>(residual + base + c, res[i]);
    }
  }
  const float s = post ? inv_rms<L, I, V>(v, C, eps) : 1.f;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * L) * V;
    if (live && c < C) {
      float g[V];
#pragma unroll
      for (int e = 0; e < V; ++e) g[e] = 1.f;
      if (gate) {
        load_vec<T, V>(gate + base + c, g);
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = activate<T>(g[e], act);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = v[i][e];
        if (post) u = u * s * post[c + e];
        u *= g[e];
        if (scale) u *= scale[c + e];
        v[i][e] = res[i][e] + alpha * u;
      }
      if (residual_out) store_vec<T, V>(residual_out + base + c, v[i]);
    }
  }
  const float q = inv_rms<L, I, V>(v, C, eps);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * L) * V;
    if (c < C) {
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = v[i][e] * q * weight[c + e];
      store_vec<T, V>(y + base + c, o);
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
  else if (n <= 128) KDA_ROW(64, 2);
  else if (n <= 256) KDA_ROW(256, 1);
  else if (n <= 512) KDA_ROW(256, 2);
  else if (n <= 1024) KDA_ROW(256, 4);
  else if (V > 4 || n <= 2048) KDA_ROW(1024, 2);
  else if (V > 1 || n <= 4096) KDA_ROW(1024, 4);
  else KDA_ROW(1024, 16);
#undef KDA_ROW
}
static_assert(KDA_NORM_MAX <= 1024 * 2 * 8 && KDA_NORM_MAX <= 1024 * 4 * 4 && KDA_NORM_MAX <= 1024 * 16, "longest rows");

template <typename T, int V>
void gated_t(const GatedNormArgs& a) {
  const int64_t rows = (int64_t)a.T * a.H;
  by_length<V>((a.D + V - 1) / V, [&](auto L, auto I) {
    constexpr int l = decltype(L)::value, i = decltype(I)::value, per = threads_of<l>() / l;
    hipLaunchKernelGGL((gated_norm_kernel<T, V, l, i>), dim3((unsigned)((rows + per - 1) / per)),
                       dim3(threads_of<l>()), 0, a.stream, (const T*)a.x, a.x_stride, (const T*)a.gate, a.gate_stride,
                       a.weight, a.weight_per_head, rows, a.H, a.D, a.act, a.gate_first, a.eps, (T*)a.y);
  });
}
template <typename T, int V>
void residual_t(const ResidualNormArgs& a) {
  by_length<V>((a.C + V - 1) / V, [&](auto L, auto I) {
    constexpr int l = decltype(L)::value, i = decltype(I)::value, per = threads_of<l>() / l;
    hipLaunchKernelGGL((residual_norm_kernel<T, V, l, i>), dim3((unsigned)(((int64_t)a.T + per - 1) / per)),
                       dim3(threads_of<l>()), 0, a.stream, (const T*)a.x, (const T*)a.residual, (const T*)a.gate,
                       a.weight, a.post_weight, a.scale, (int64_t)a.T, a.C, a.act, a.alpha, a.eps, (T*)a.residual_out,
                       (T*)a.y);
  });
}

int64_t row_threads(int64_t rows, int n, int v) {
  int64_t t = 0;
  auto f = [&](auto L, auto) { t = (rows + 255) * decltype(L)::value; };
  if (v == 8) by_length<8>(n, f);
  else if (v == 4) by_length<4>(n, f);
  else by_length<1>(n, f);
  return t;
}
int width_of(const GatedNormArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  return a.D % v == 0 && a.x_stride % v == 0 && (!a.gate || a.gate_stride % v == 0) ? v : 1;
}
int width_of(const ResidualNormArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  return a.C % v == 0 ? v : 1;
}

}  // namespace

int64_t gated_threads(const GatedNormArgs& a) {
  const int v = width_of(a);
  return row_threads((int64_t)a.T * a.H, (a.D + v - 1) / v, v);
}
int64_t residual_threads(const ResidualNormArgs& a) {
  const int v = width_of(a);
  return row_threads(a.T, (a.C + v - 1) / v, v);
}

hipError_t launch_gated_norm(const GatedNormArgs& a) {
  const bool vec = width_of(a) > 1;
  if (a.bf16) vec ? gated_t<bf16_bits, 8>(a) : gated_t<bf16_bits, 1>(a);
  else vec ? gated_t<float, 4>(a) : gated_t<float, 1>(a);
  return hipGetLastError();
}

hipError_t launch_residual_norm(const ResidualNormArgs& a) {
  const bool vec = width_of(a) > 1;
  if (a.bf16) vec ? residual_t<bf16_bits, 8>(a) : residual_t<bf16_bits, 1>(a);
  else vec ? residual_t<float, 4>(a) : residual_t<float, 1>(a);
  return hipGetLastError();
}

}  // namespace kda
