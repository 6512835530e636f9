// 8-bit cache of recurrent states on gfx950: blocks of 32 consecutive values
// share a power-of-two step 2^e, e the least with max|x| <= qmax 2^e.
//
// The step is a power of two so that scaling is exact in both directions: the
// only rounding is the one to 8 bits, and a store rounds the same way whatever
// computes it. Both kernels are bound by memory, 5.03 D^2 bytes per head: 256 x
// 32 heads stored in 122 us (5.5 TB/s) and loaded in 98 to 112 us (6.0 to 6.9).
#include "kda_device.h"
#include "kda_internal.h"

#include <float.h>

namespace kda {

constexpr int kBlock = KDA_CACHE_BLOCK;

// e + 127 for a block whose largest finite magnitude is amax. amax = m 2^x with
// m in [1, 2): qmax = 1.984375 2^6 (int8) or 1.75 2^8 (e4m3), so
// e = x - 6 (or x - 8), one more if m lies above. Subnormal amax and results
// below -127 take -127.
template <bool kE4m3>
__device__ __forceinline__ int step_code(float amax) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, amax);
  const uint32_t edge = kE4m3 ? 0x600000u : 0x7e0000u;   // mantissa bits of 1.75, 1.984375
  const int code = (int)(bits >> 23) - (kE4m3 ? 8 : 6) + ((bits & 0x7fffffu) > edge ? 1 : 0);
  return max(code, 0);
}

__device__ __forceinline__ bool finite(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7f800000u) != 0x7f800000u;
}

// Four values scaled by 2^-e and rounded to 8 bits each.
template <bool kE4m3>
__device__ __forceinline__ uint32_t pack4(f32x4 x, int code) {
  constexpr float top = kE4m3 ? 448.f : 127.f;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = __builtin_amdgcn_ldexpf(x[i], 127 - code);
    // infinities become the largest value; NaN is kept (e4m3) or 0 (int8)
    const bool nan = x[i] != x[i];
    y[i] = fminf(fmaxf(y[i], -top), top);
    if (nan) y[i] = kE4m3 ? x[i] : 0.f;
  }
  if constexpr (kE4m3) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], r, true);
  } else {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= ((uint32_t)(int)rintf(y[i]) & 0xffu) << (8 * i);
    return r;
  }
}

template <bool kE4m3>
__device__ __forceinline__ f32x4 unpack4(uint32_t w, int code) {
  f32x4 y;
  if constexpr (kE4m3) {
    y[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
    y[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
    y[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
    y[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (float)(int8_t)(w >> (8 * i));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a value next to the largest float may have been rounded up past it
    y[i] = __builtin_amdgcn_ldexpf(y[i], code - 127);
    y[i] = y[i] > FLT_MAX ? FLT_MAX : y[i] < -FLT_MAX ? -FLT_MAX : y[i];
  }
  return y;
}

// One workgroup per (state, head). Lane l of a wave takes four consecutive
// values, eight lanes a block.
template <int D, bool kE4m3>
__global__ __launch_bounds__(D == 128 ? 256 : 64) void cache_store_kernel(
    const float* __restrict__ states, const int32_t* __restrict__ slots, uint32_t* __restrict__ values,
    uint8_t* __restrict__ scales, int N, int num_slots, int H) {
  constexpr int kThreads = D == 128 ? 256 : 64;
  constexpr int kIters = D * D / 4 / kThreads;
  const uint32_t n = blockIdx.x / (uint32_t)H, h = blockIdx.x % (uint32_t)H;
  const int tid = threadIdx.x;
  const int slot = slots ? slots[n] : (int)n;
  if (slot < 0 || slot >= num_slots) return;
  const f32x4* src = (const f32x4*)(states + (size_t)blockIdx.x * D * D);
  f32x4 x[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) x[i] = __builtin_nontemporal_load(src + tid + i * kThreads);
  if (slots && n + 1 < (uint32_t)N) {   // a later state of the same slot is the one that is written
    // kScan loads in flight, those past the end of the last entry (a later
    // state's too): 16384 states of 128 x 128 in 252 us, 311 with one at a time,
    // 223 without a list. Every head of every state looks through the rest of the
    // list, N^2 H / 2 reads: 65536 states of 8 heads of 16 x 16 take 2944 us, 117
    // without a list.
    constexpr int kScan = 8;
    int later = 0;
    for (int m = (int)n + 1 + tid; m < N; m += kScan * kThreads) {
      int other[kScan];
#pragma unroll
      for (int j = 0; j < kScan; ++j) other[j] = slots[min(m + j * kThreads, N - 1)];
#pragma unroll
      for (int j = 0; j < kScan; ++j) later |= other[j] == slot;
    }
    if (__syncthreads_or(later)) return;
  }
  const size_t dst = (size_t)slot * H + h;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) amax = fmaxf(amax, finite(x[i][c]) ? fabsf(x[i][c]) : 0.f);
    amax = fmaxf(amax, lane_xor<1>(amax));
    amax = fmaxf(amax, lane_xor<2>(amax));
    amax = fmaxf(amax, lane_xor<4>(amax));
    const int code = step_code<kE4m3>(amax);
    const int e = tid + i * kThreads;
    values[dst * (D * D / 4) + e] = pack4<kE4m3>(x[i], code);
    if (tid % 8 == 0) scales[dst * (D * D / kBlock) + e / 8] = (uint8_t)code;
  }
}

template <int D, bool kE4m3>
__global__ __launch_bounds__(D == 128 ? 256 : 64) void cache_load_kernel(
    const uint32_t* __restrict__ values, const uint8_t* __restrict__ scales, const int32_t* __restrict__ slots,
    float* __restrict__ states, int num_slots, int H) {
  constexpr int kThreads = D == 128 ? 256 : 64;
  constexpr int kIters = D * D / 4 / kThreads;
  const uint32_t n = blockIdx.x / (uint32_t)H, h = blockIdx.x % (uint32_t)H;
  const int tid = threadIdx.x;
  const int slot = slots ? slots[n] : (int)n;
  f32x4* dst = (f32x4*)(states + (size_t)blockIdx.x * D * D);
  if (slot < 0 || slot >= num_slots) {
#pragma unroll
    for (int i = 0; i < kIters; ++i) __builtin_nontemporal_store(f32x4{0.f, 0.f, 0.f, 0.f}, dst + tid + i * kThreads);
    return;
  }
  const size_t src = (size_t)slot * H + h;
  uint32_t w[kIters];
  int code[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int e = tid + i * kThreads;
    w[i] = values[src * (D * D / 4) + e];
    code[i] = scales[src * (D * D / kBlock) + e / 8];
  }
#pragma unroll
  for (int i = 0; i < kIters; ++i)
    __builtin_nontemporal_store(unpack4<kE4m3>(w[i], code[i]), dst + tid + i * kThreads);
}

template <int D, bool kE4m3>
static hipError_t launch_cache_t(const CacheArgs& a, bool store) {
  const dim3 grid((unsigned)((int64_t)a.N * a.H)), block(D == 128 ? 256 : 64);
  if (store)
    hipLaunchKernelGGL((cache_store_kernel<D, kE4m3>), grid, block, 0, a.stream, a.states, a.slots,
                       (uint32_t*)a.values, a.scales, a.N, a.num_slots, a.H);
  else
    hipLaunchKernelGGL((cache_load_kernel<D, kE4m3>), grid, block, 0, a.stream, (const uint32_t*)a.values,
                       a.scales, a.slots, a.states, a.num_slots, a.H);
  return hipGetLastError();
}

static hipError_t launch_cache(const CacheArgs& a, bool store) {
  if (a.D == 128) return a.e4m3 ? launch_cache_t<128, true>(a, store) : launch_cache_t<128, false>(a, store);
  return a.e4m3 ? launch_cache_t<16, true>(a, store) : launch_cache_t<16, false>(a, store);
}
hipError_t launch_cache_store(const CacheArgs& a) { return launch_cache(a, true); }
hipError_t launch_cache_load(const CacheArgs& a) { return launch_cache(a, false); }

}  // namespace kda
