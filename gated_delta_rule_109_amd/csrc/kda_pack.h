// Device-side helpers of the calls around a recurrence (convolution, scan,
// norms): vectors of elements, activations, and where a workgroup's tokens lie
// in packed sequences.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// V consecutive elements, as one load or store of up to 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[V]) {
  const Pack<T, V> v = *(const Pack<T, V>*)p;
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = Elem<T>::load(&v.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
  Pack<T, V> v;
#pragma unroll
  for (int i = 0; i < V; ++i) Elem<T>::store(&v.e[i], x[i]);
  *(Pack<T, V>*)p = v;
}

// 1 / (1 + e^-x). bf16 outputs: hardware exp2 and reciprocal, a few units of
// 2^-23, far below their rounding. fp32 outputs: within about 2^-23.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * kLog2e));
  else return 1.0f / (1.0f + expf(-x));
}
template <typename T>
__device__ __forceinline__ float activate(float x, int act) {
  if (act == KDA_ACT_NONE) return x;
  const float s = sigmoid<T>(x);
  return act == KDA_ACT_SILU ? x * s : s;
}

// Part j of a packed sequence cut every `len` tokens.
struct Part {
  int n, j, parts;    // sequence, part of it, parts it has (at least 1)
  int first, count;   // its tokens (none: an empty sequence)
  int start, length;  // the sequence's tokens
};
// First token of sequence n (n = num_seqs: the end), inside [0, T] whatever
// the offsets hold.
__device__ __forceinline__ int token_offset(const Packed& s, int n) {
  return s.cu ? min(max(s.cu[n], 0), s.T) : n * s.T;
}
// Parts are numbered without a table: part j of sequence n is slot
// offset(n) / len + n + j. A sequence of L tokens has max(1, ceil(L / len))
// parts, at most offset(n + 1) / len - offset(n) / len + 1, so slots never
// collide and there are at most T / len + num_seqs. False: no part has this slot.
__device__ __forceinline__ bool find_part(const Packed& s, int len, int slot, Part& p) {
  int lo = 0, hi = s.num_seqs;   // the last n in [lo, hi) whose first slot is at most `slot`
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (token_offset(s, mid) / len + mid <= slot) lo = mid;
    else hi = mid;
  }
  p.n = lo;
  p.start = token_offset(s, lo);
  p.length = max(token_offset(s, lo + 1) - p.start, 0);
  p.j = slot - (p.start / len + lo);
  p.parts = p.length ? (p.length - 1) / len + 1 : 1;
  if (p.j < 0 || p.j >= p.parts) return false;
  p.first = p.start + p.j * len;
  p.count = min(len, p.length - p.j * len);
  return true;
}
inline int64_t part_slots(const Packed& s, int len) { return (int64_t)s.T / len + s.num_seqs; }

}  // namespace kda
