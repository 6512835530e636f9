// Device-side helpers of the calls around a recurrence (convolution, scan,
// norms): vectors of elements, activations, and where a workgroup's tokens lie
// in packed sequences.
#pragma once

#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

// V consecutive elements as one load or store, at the elements' own alignment
// (gfx950's global accesses need no more).
template <typename T, typename W>
struct Unaligned {
  typedef W type __attribute__((aligned(sizeof(T))));
};
template <typename T, int V>
struct Bits {
  static_assert(sizeof(T) * V == 16 || sizeof(T) * V == 8, "8 or 16 bytes");
  typedef uint32_t type __attribute__((ext_vector_type(sizeof(T) * V / 4)));
  typedef typename Unaligned<T, type>::type unaligned;
};
template <typename T, int V>
using bits_t = typename Bits<T, V>::type;
template <typename T, int V>
__device__ __forceinline__ bits_t<T, V> load_bits(const T* p) {
  return *(const typename Bits<T, V>::unaligned*)p;
}
// Outputs go past the caches (a prompt's are larger than they are, and who reads
// them runs on other dies: a convolution of 8192 x 12288 bf16 over and over 92 -> 73
// us; one of 3001 x 777 fp32 takes the same either way).
template <typename T, int V>
__device__ __forceinline__ void store_bits(T* p, bits_t<T, V> v) {
  __builtin_nontemporal_store(v, (typename Bits<T, V>::unaligned*)p);
}
template <typename T, int V>
__device__ __forceinline__ void from_bits(bits_t<T, V> v, float (&out)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 4) out[i] = __uint_as_float(v[i]);
    else out[i] = __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
  }
}
template <typename T, int V>
__device__ __forceinline__ bits_t<T, V> to_bits(const float (&x)[V]) {
  bits_t<T, V> v;
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) {
    if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(x[i]);
    else v[i] = (uint32_t)f32_to_bf16_bits(x[2 * i]) | (uint32_t)f32_to_bf16_bits(x[2 * i + 1]) << 16;
  }
  return v;
}
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&out)[V]) {
  from_bits<T, V>(load_bits<T, V>(p), out);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[V]) {
  store_bits<T, V>(p, to_bits<T, V>(x));
}
// Vector i of a row. Of a row that is not whole vectors the last one is its last V
// elements, of which the vector in front has the first `skip`: they are read as well,
// which takes one load and no branch, and not written (with its end read by single
// elements a residual norm of 8192 x 4097 bf16 took 131 us, not 88, a convolution 50,
// not 39). Rows shorter than a vector: element by element.
template <int V, bool whole>
struct VecAt {
  int c, skip;      // first element
  bool on;          // the row has this vector
  // Element e belongs to this vector of the row.
  __device__ __forceinline__ bool owns(int e, int width) const { return whole ? on : e >= skip && c + e < width; }
};
template <int V, bool whole>
__device__ __forceinline__ VecAt<V, whole> vec_at(int i, int width) {
  const int c = i * V, over = c + V - width;
  const bool shift = !whole && over > 0 && width >= V;
  return {shift ? width - V : c, shift ? over : 0, c < width};
}
template <bool whole, typename T, int V>
__device__ __forceinline__ bits_t<T, V> load_row(const T* p, int width) {
  if (whole || width >= V) return load_bits<T, V>(p);
  bits_t<T, V> v = {};
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (i < width) {
      if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(p[i]);
      else v[i / 2] |= (uint32_t)p[i] << (i % 2 ? 16 : 0);
    }
  return v;
}
// The last n of V elements, n < V: in runs of V / 2, V / 4, .. as n has them.
template <typename T, int V>
__device__ __forceinline__ void store_last(T* p, bits_t<T, V> v, int n) {
  constexpr int D = V * sizeof(T) / 4;                   // dwords
  typedef uint32_t two __attribute__((ext_vector_type(2)));
  static_assert(D == 4, "16 bytes");
  const int m = n * (int)sizeof(T);                      // bytes
  if (m & 8) __builtin_nontemporal_store(two{v[2], v[3]}, (typename Unaligned<T, two>::type*)((char*)p + 8));
  const int q = m & 8 ? 1 : 3;                           // dword in front of those
  if (m & 4) __builtin_nontemporal_store(m & 8 ? v[1] : v[3], (typename Unaligned<T, uint32_t>::type*)((char*)p + 4 * q));
  if constexpr (sizeof(T) == 2)
    if (m & 2) {
      const int d = 3 - (m >> 2);
      p[2 * d + 1] = (T)((d > 1 ? d > 2 ? v[3] : v[2] : d ? v[1] : v[0]) >> 16);
    }
}
template <bool whole, typename T, int V>
__device__ __forceinline__ void store_row(T* p, bits_t<T, V> v, int skip, int width) {
  if (whole || width >= V) {
    if (whole || skip == 0) store_bits<T, V>(p, v);
    else store_last<T, V>(p, v, V - skip);
    return;
  }
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (i < width) {
      if constexpr (sizeof(T) == 4) p[i] = __uint_as_float(v[i]);
      else p[i] = (T)(i % 2 ? v[i / 2] >> 16 : v[i / 2]);
    }
}
// The first n of V fp32 parameters (`fill` for the others).
template <int V>
__device__ __forceinline__ void load_params(const float* p, int n, float fill, float (&out)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    if (n >= i + 4) {
      const bits_t<float, 4> v = load_bits<float, 4>(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[i + e] = __uint_as_float(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[i + e] = i + e < n ? p[i + e] : fill;
    }
  }
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
// The last sequence n with offset(n) / len + n * each <= at (0: there is none) and its
// tokens, found by a whole wave: each step looks at 64 places at once (a step is a
// load's latency, and a prompt of a few sequences takes microseconds), and the last
// one has loaded what the sequence begins and ends at.
__device__ __forceinline__ int last_sequence(const Packed& s, int len, int each, int at, int& start, int& end) {
  if (s.num_seqs == 1) {
    start = token_offset(s, 0), end = token_offset(s, 1);
    return 0;
  }
  const int lane = threadIdx.x % kWave;
  int lo = 0, n = s.num_seqs;            // it is in [lo, lo + n)
  while (n > kWave) {
    const int step = (n + kWave - 1) / kWave, d = lane * step;
    const bool below = d < n && token_offset(s, lo + min(d, n - 1)) / len + (lo + d) * each <= at;
    const int last = max(__popcll(__ballot(below)) - 1, 0) * step;
    lo += last;
    n = min(step, n - last);
  }
  const int offset = token_offset(s, lo + min(lane, n));
  const int i = max(__popcll(__ballot(lane < n && offset / len + (lo + lane) * each <= at)) - 1, 0);
  start = __builtin_amdgcn_readlane(offset, i);
  end = i + 1 < kWave ? __builtin_amdgcn_readlane(offset, i + 1) : token_offset(s, lo + kWave);
  return __builtin_amdgcn_readfirstlane(lo + i);
}
// Parts are numbered without a table: part j of sequence n is slot
// offset(n) / len + n + j. A sequence of L tokens has max(1, ceil(L / len))
// parts, at most offset(n + 1) / len - offset(n) / len + 1, so slots never
// collide and there are at most T / len + num_seqs. False: no part has this slot.
// (All threads of a wave ask together.)
__device__ __forceinline__ bool find_part(const Packed& s, int len, int slot, Part& p) {
  int end;
  p.n = last_sequence(s, len, 1, slot, p.start, end);
  p.length = max(end - p.start, 0);
  p.j = slot - (p.start / len + p.n);
  p.parts = p.length ? (p.length - 1) / len + 1 : 1;
  if (p.j < 0 || p.j >= p.parts) return false;
  p.first = p.start + p.j * len;
  p.count = min(len, p.length - p.j * len);
  return true;
}
inline int64_t part_slots(const Packed& s, int len) { return (int64_t)s.T / len + s.num_seqs; }

}  // namespace kda
