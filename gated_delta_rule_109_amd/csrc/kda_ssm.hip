// Selective state-space scan over packed sequences on gfx950, for prompts and
// for single tokens (kda.h: kda_ssm_prefill, kda_ssm_step).
//
//   S_t = exp(d_t a) S_{t-1} + d_t b_t x_t^T,   y_t = S_t^T c_t + skip x_t
//
// One decay per head and token; S is N x P in fp32. Prompts run in chunks on the
// matrix cores.
#include "kda_pack.h"

#include <math.h>

#include <algorithm>

namespace kda {
namespace {

constexpr int kThreads = 256;

// Segments. A call with few sequences, heads and columns cuts its sequences
// every segment_len tokens, and the segments run side by side in three launches:
//   1: every segment but the last of its sequence, for its last state alone: the
//      first from the initial state, the others from 0.
//   2: the states in front of the segments, in order:
//      front(j + 1) = e^{sum of d a over segment j} front(j) + last state of segment j.
//   3: every segment from the state in front of it, with its outputs.
// Final states may replace the initial ones: where they do, the first launch keeps
// a copy for the first segment of the third. The state in front of segment j of a
// sequence that starts at token s is entry 2 (s / len) + j: a sequence of two or
// more segments reaches over at least one multiple of len, and has at most one
// segment more than it reaches over, so no two meet and there are 2 T / len.
//
// How long is estimated from what was measured (by `cost` below, in us): a chunk of both
// launches takes its time on the chain of a segment's chunks, more of it where compute
// units hold two workgroups or more; a segment adds its state, written and read twice,
// and a step of the chain of its sequence's states. Compared are the lengths that fill
// one and two rounds of workgroups, the least one that the target allows (at least
// twice the average sequence where sequences alone fill the GPU), and those where
// chain and segments balance. The constants are fitted by hand to measured calls: over 38
// of 700 to 8192 tokens the length taken is on average 2.9 % slower than the best one, at
// most 14 % (2048 tokens of six sequences, 20 heads 128 x 128 fp32: 97 us, 85 by longer
// segments). Calls of few tokens are not split: 300 tokens of two sequences whole 13 us,
// in segments 19.
struct Split {
  int columns;     // columns of a head one workgroup owns
  int target;      // workgroups that the segments of a call make up, sequences' rests aside
  int chunk;       // tokens: segments are whole chunks, at least two
  int whole;       // calls of at most so many tokens are not split
};
// (the chunks' workgroups have 8 waves where a head has more than 64 columns, else 4.
// Of states of 256 rows a compute unit holds one workgroup, where more of them run in
// turns: 8192 tokens of 16 heads 256 x 128 in one round 108 us; when outputs had two terms
// of S and M it took 100, and two rounds 153. Of smaller states it holds two and more; 3
// or 4 for 64 columns gained nothing then: 32 heads of 16 x 64 49 us, with 1024
// workgroups 54)
enum Kind { kF32, kNarrow, kWide };
Split split_of(Kind k, int N) {
  const int target = N == 256 ? 256 : 512;
  if (k == kF32) return {64, target, 32, 160};
  return {k == kWide ? 128 : 64, target, KDA_SSM_CHUNK, 384};
}
Split split_of(bool bf16, int N, int P) { return split_of(!bf16 ? kF32 : P <= 64 ? kNarrow : kWide, N); }
int column_blocks(const Split& s, int P) { return (P + s.columns - 1) / s.columns; }

int segment_len(const Packed& s, int H, int N, int P, const Split& sp) {
  const int64_t groups = (int64_t)H * column_blocks(sp, P);   // workgroups a segment
  const int64_t parts = sp.target / groups;                   // segments of all sequences together
  if (parts < 2 || s.T <= sp.whole) return s.T > 0 ? s.T : 1;
  constexpr int kUnits = 256;
  const double chunks = (double)s.T / sp.chunk, n = s.num_seqs > 1 ? s.num_seqs : 1;
  const double chunk_us = sp.chunk == KDA_SSM_CHUNK ? 2 + N / 40.0 : 1.7 + N / 32.0;
  const double segment_us = 0.35 / sqrt(n) + 1.4 * H * N * P / (1 << 19);
  const double ends = n > 1 ? 0.6 * n : 0;                    // segments that are a sequence's rest
  auto cost = [&](int64_t k) {                                // segments of k chunks
    const double count = n > 1 ? std::max(chunks / k + ends, n) : ceil(chunks / k), held = count * groups / kUnits;
    return chunk_us * k * (held <= 1 ? 1 : std::max(1.4, 0.8 * held)) + segment_us * chunks / k;
  };
  int64_t least = std::max<int64_t>(2, (int64_t)ceil(chunks / parts));
  if (n * groups >= 0.9 * sp.target) least = std::max<int64_t>(least, (int64_t)ceil(2 * chunks / n));
  const int64_t even = (int64_t)sqrt(segment_us * chunks / chunk_us);
  int64_t best = least;
  auto consider = [&](int64_t k) {
    if (k > least && cost(k) < cost(best)) best = k;
  };
  consider(even);
  consider(even + 1);
  for (int rounds = 1; rounds <= 2; ++rounds) {
    const double room = n > 1 ? (double)rounds * kUnits / groups - ends : (double)(rounds * kUnits / groups);
    if (room >= 1) consider((int64_t)ceil(chunks / room));
  }
  return (int)(best * sp.chunk);
}

// d_t of one token and head.
__device__ __forceinline__ float step_size(float dt, float bias, bool softplus) {
  const float v = dt + bias;
  // ln(1 + e^v) = max(v, 0) + ln(1 + e^-|v|); NaN stays NaN
  return softplus ? (v > 0.f ? v : v < 0.f ? 0.f : v) + log1pf(expf(-fabsf(v))) : v;
}

// A factor e^x in two, so that it does not overflow before what it multiplies has its say:
// e^min(x, kMostGrowth), and with x above that e^(x - kMostGrowth) besides, which leaves a
// state of 0 at 0 whatever it is.
constexpr float kMostGrowth = 88.f;
__device__ __forceinline__ f32x4 grown(f32x4 s, float x) {
  const float f = expf(x - kMostGrowth);
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = s[i] == 0.f ? 0.f : s[i] * f;
  return s;
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
  bool keep;        // final states replace the initial ones
  float* ends;      // states in front of segments [entry][H][P blocks][..]
  double* sums;     // sum of d a over a segment, at the entry in front of it [entry][H]
};
__device__ __forceinline__ size_t entry_of(const SsmParams& a, const Part& p, int h, int j) {
  return (size_t)(2 * (p.start / a.len) + j) * a.H + h;
}
// State in front of segment j, `vecs` vectors for each column block.
__device__ __forceinline__ f32x4* front_of(const SsmParams& a, const Part& p, int h, int j, int pblocks, int pb,
                                           int vecs) {
  return (f32x4*)a.ends + (entry_of(a, p, h, j) * pblocks + pb) * (size_t)vecs;
}

// ---- bf16: chunks of 64 tokens on the matrix cores --------------------------------------
//
// With c_t = sum of d a up to token t of the chunk and S the state in front of it:
//     y_t = e^{c_t} C_t^T S + sum_{s <= t} M[t][s] x_s,  M[t][s] = e^{c_t - c_s} d_s (C_t . B_s), M[t][t] += skip
//     S  <- e^{c_L} S + sum_s B_s (w_s x_s)^T,           w_s = e^{c_L - c_s} d_s
// B, C and x are bf16 and enter the products as they are. The fp32 factor of
// each product (S, M and w x) is split into three bf16 terms, which hold its 24 bits.
// (With two of S and M a call of 8192 tokens of 32 heads took 114 us, not 125, but its
// outputs were off by 2^-17 of each product, which shows where products cancel.) Sums of
// d a are taken in fp64 and handed on as two floats, so that their differences are exact
// to fp32.
//
// A workgroup owns 16 W columns of a head, wave w the 16 columns from 16 w on,
// with their whole state in accumulators: tile k holds rows 16 k + 4 g
// + i of column l % 16 (l the lane, g = l / 16). As operand of the next product a
// lane holds 8 values along the sum: taking rows 16 (2v) + 4g + i and
// 16 (2v + 1) + 4g + i for them makes the accumulators of two tiles that operand
// without a move. The other operands are read in the same order:
//   sC, sB  [token][channel], sX [token][column]: as they come, but channel 32 v +
//        16 u + 4 g + i of a row is kept at 32 v + 8 g + 4 u + i, so that an operand
//        of sums over channels is one read of 16 bytes. Sums over tokens read 4 rows
//        of 16 columns turned over (a lane: one column, 4 tokens), twice an operand.
//   sM   [term][token t][token s], s kept in the order of the channels
// No padding: blocks of 16 bytes are XORed with bits of their row, so that the
// lanes an LDS instruction serves at a time meet different banks: 16 rows at one
// block (16 bytes a lane: lanes 0-3, 12-15, 20-23, 24-27 and so on), and 4 rows of
// 16 columns (turned over: 16 lanes).
//
// 8192 tokens of 32 heads 128 x 128: states 34 us, fronts 13, outputs 84, where the
// bytes take 32 (copies reach 5.35 TB/s) and the products as written 36 (120 a chunk
// and wave in the outputs' launch, 48 in the other). Neither bounds it: four waves a
// SIMD wait for each other at three barriers a chunk. With two terms of S and M, when
// the outputs took 73 to 77, matrix instructions, vector instructions and LDS were at
// work for about 20, 30 and 28 us of them; a third workgroup a compute unit (M in the
// place of C, 64 columns) changed nothing; scaling the state as it is split, and reads of
// LDS held ahead of the work that hides them, spilled (80 and 73 to 77 us); w x in two
// terms where only outputs come of the state gained 2 us.
constexpr int kL = KDA_SSM_CHUNK;

// Workgroups go to the 8 dies in turn. They are numbered so that kShare of those that
// share B and C (a group's heads in a segment) are on one die and meet in its L2; not
// more, or a few segments of many heads leave dies without work (8192 tokens of 128
// heads 128 x 64 in one group: eight 233 us; with outputs of two terms of S and M 220,
// and all of a segment on a die 419).
constexpr int kDies = 8, kShare = 8;
__host__ __device__ __forceinline__ int shared_groups(int heads, int blocks) {
  return (int64_t)heads * blocks < kShare ? heads * blocks : kShare;
}
__device__ __forceinline__ int numbered(int share) {
  return (blockIdx.x / (kDies * share) * kDies + blockIdx.x % kDies) * share + blockIdx.x / kDies % share;
}

// Block b of row 16 k + l is kept at b ^ row_mask(l), by the row's bf16 elements. A
// lane keeps one place in each array; others are that one XOR a constant (other
// blocks) plus a constant (other tiles). The mask: rows 4 j' + j of one j' in
// different fours of blocks (as far as those are not different banks anyway), and
// 0, 2, 3, 1 by j' in the four: { m(0), m(3), m(1) ^ 1, m(2) ^ 1 } are all of it.
template <int NP>
__device__ __forceinline__ constexpr int row_mask(int l) {
  const int m = (l >> 2 & 1) << 1 ^ (l >> 3) * 3;
  return NP >= 128 ? (l & 3) << 2 | m : NP == 64 ? (l >> 1 & 1) << 2 | m : m;
}
// Place in a row (row l of its tile) of channels 8 nv .. 8 nv + 7: the first four, in
// one block; the others are in the next one.
template <int NP>
__device__ __forceinline__ int channel_place(int nv, int l) {
  return (4 * (nv / 4) + 2 * (nv & 1) ^ row_mask<NP>(l)) * 8 + 4 * (nv / 2 & 1);
}
__device__ __forceinline__ void store_channels(bf16_bits* dst, int place, u32x4 v) {
  *(uint2*)(dst + place) = uint2{v[0], v[1]};
  *(uint2*)(dst + (place ^ 8)) = uint2{v[2], v[3]};
}
// 16 lanes, each with the place of 4 elements (lanes 4 j .. 4 j + 3: row j of 4, 16
// columns): lane l gets column l of the 4 rows.
__device__ __forceinline__ bf16x4 read_turned(const bf16_bits* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds;
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds*)p));
}
// v, and the compiler does not know it: what is made of it is made where it is
// used, not once and kept in registers (which spill).
template <typename T>
__device__ __forceinline__ T fresh(T v) {
  asm volatile("" : "+v"(v));
  return v;
}

// What is the same in all lanes.
__device__ __forceinline__ float uniform(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
// Keeps an array in scratch memory.
template <typename T>
__device__ __forceinline__ void in_memory(T* p) {
  asm volatile("" ::"v"((__attribute__((address_space(5))) T*)p) : "memory");
}
// The value of lane `l` (its low 6 bits).
__device__ __forceinline__ double lane_value(double x, int l) {
  const uint2 v = __builtin_bit_cast(uint2, x);
  return __builtin_bit_cast(double, make_uint2(__builtin_amdgcn_ds_bpermute(4 * l, v.x),
                                               __builtin_amdgcn_ds_bpermute(4 * l, v.y)));
}

// x - h, h bf16 terms of x: exact, and one instruction a value, the sum of
// products of a pair of bf16 with (-1, 0) or (0, -1), where the pair taken apart takes
// two (8192 tokens of 32 heads: states 35.0 -> 33.7 us, outputs 76.8 -> 75.0). The factors come from registers: as
// an instruction's own constant, -1 stands in the wrong half of its pair.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
struct Minus {
  bf16x2 lo, hi;
};
__device__ __forceinline__ Minus minus_one() {
  uint32_t lo = 0xbf80u, hi = 0xbf800000u;
  asm("" : "+s"(lo), "+s"(hi));
  return {__builtin_bit_cast(bf16x2, lo), __builtin_bit_cast(bf16x2, hi)};
}
__device__ __forceinline__ f32x4 rest_of(f32x4 x, bf16x4 h, const Minus& m) {
  const uint2 p = __builtin_bit_cast(uint2, h);
  const bf16x2 a = __builtin_bit_cast(bf16x2, p.x), b = __builtin_bit_cast(bf16x2, p.y);
  return f32x4{
      __builtin_amdgcn_fdot2_f32_bf16(a, m.lo, x[0], false), __builtin_amdgcn_fdot2_f32_bf16(a, m.hi, x[1], false),
      __builtin_amdgcn_fdot2_f32_bf16(b, m.lo, x[2], false), __builtin_amdgcn_fdot2_f32_bf16(b, m.hi, x[3], false)};
}
// The upper halves of four floats: bf16, rounded towards zero.
__device__ __forceinline__ bf16x4 upper_halves(f32x4 x) {
  const u32x4 v = __builtin_bit_cast(u32x4, x);
  return __builtin_bit_cast(bf16x4, uint2{__builtin_amdgcn_perm(v[1], v[0], 0x07060302u),
                                          __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)});
}
// x = h + m + l in bf16, 8 bits each, each towards zero, the rest of the ones before: exact
// (but for rests below 2^-126, which are taken as 0).
// (To nearest, as many instructions, a finite x above the largest bf16 would become
// infinite, and the rest of it NaN.)
__device__ __forceinline__ void split3(f32x4 x, bf16x4& h, bf16x4& m, bf16x4& l, const Minus& one) {
  h = upper_halves(x);
  const f32x4 r = rest_of(x, h, one);
  m = upper_halves(r);
  l = to_bf16x4(rest_of(r, m, one));
}

// What the tokens of a chunk need of d and a.
template <int L>
struct alignas(16) Decays {
  float hi[L], lo[L];   // c_t log2 e
  float d[L];           // d_t
  float e[L];           // e^{c_t}
  float w[L];           // e^{c_L - c_t} d_t
  float total;          // e^{c_L}
  int grows;            // the chunk is taken by tokens
};
// A wave's 64 tokens, one a lane (at: the lane; on: it has one): the decays of 64 / L
// chunks, with the sums of the logarithms c = d a in fp64. Returns the last chunk's c_L
// in every lane of it. One logarithm is no less than kLeast: e^kLeast and all that is
// multiplied by it are 0 as it is, while a token that ends the state (d a = -1e12)
// would take the digits of the sums behind it.
//
// Factors between tokens of a chunk that grow may overflow where the state that they
// multiply is 0 or small. Of a chunk whose growing tokens alone make more than
// kMostInChunk of a logarithm (about 2^63: as much is left for c . b d) the tokens are
// taken one after the other (8192 tokens of 32 heads 128 x 128, every chunk so: bf16 7.6
// ms, fp32 6.1).
template <int L>
__device__ __forceinline__ double make_decays(bool on, float d, float a, int at, Decays<L>* dec) {
  constexpr double kLeast = -(1 << 20), kMostInChunk = 44.0;
  double c = on ? (double)d * a : 0.0;                   // (an infinite a times the d of no token: NaN)
  c = c < kLeast ? kLeast : c;                           // (NaN stays)
  int grows = 0;
  if (__any(c > 0.0)) {
    double up = c > 0.0 ? c : 0.0;
#pragma unroll
    for (int m = 1; m < L; m *= 2) up += lane_value(up, at ^ m);
    grows = up > kMostInChunk;
  }
#pragma unroll
  for (int m = 1; m < L; m *= 2) {
    const double o = lane_value(c, at - m);
    if (at % L >= m) c += o;
  }
  const double end = lane_value(c, at | (L - 1));
  constexpr double kL2 = 1.4426950408889634;
  const float hi = (float)(c * kL2);
  Decays<L>& q = dec[at / L];
  q.hi[at % L] = hi;
  q.lo[at % L] = (float)(c * kL2 - hi);
  q.d[at % L] = d;
  q.e[at % L] = __builtin_amdgcn_exp2f(hi);
  q.w[at % L] = __builtin_amdgcn_exp2f((float)((end - c) * kL2)) * d;
  if (at % L == 0) q.total = __builtin_amdgcn_exp2f((float)(end * kL2)), q.grows = grows;
  return end;
}

// Waves a SIMD that the registers leave room for: those of two workgroups a compute unit
// (of states of 256 rows, with outputs, one), and in the launches for states, which need
// less of LDS, as many as there.
constexpr int waves_of(int N, int W, bool outputs) { return outputs ? (N == 256 ? W / 4 : W / 2) : (N == 256 ? 2 : 4); }

template <int N, int W, bool outputs>
__global__ __launch_bounds__(64 * W, waves_of(N, W, outputs)) void ssm_chunk_kernel(SsmParams a) {
  constexpr int kThreads = 64 * W, kCols = 16 * W, NP = N < 32 ? 32 : N, KS = NP / 32, NT = N / 16, NV = N / 8;
  const int pblocks = (a.P + kCols - 1) / kCols;
  const int id = numbered(shared_groups(a.H / a.G, pblocks));
  const int pb = id % pblocks, h = id / pblocks % a.H;
  Part p;
  if (!find_part(a.seqs, a.len, id / pblocks / a.H, p)) return;
  const bool last = p.j == p.parts - 1;
  if (!outputs && last) return;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, g = lane / 16, l16 = lane % 16;
  const int wcol = wave * 16;                       // first column of the wave in the workgroup's
  const int col0 = pb * kCols;                           // and of the workgroup in the head
  const int grp = h / (a.H / a.G);
  const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.skip ? a.skip[h] : 0.f;

  __shared__ __attribute__((aligned(16))) bf16_bits sC[kL * NP], sB[kL * NP], sX[kL * kCols], sM[3][kL * kL];
  __shared__ Decays<kL> dec[4];

  // ---- state in front of the segment
  f32x4 s[NT];
  auto front = [&](int j) { return front_of(a, p, h, j, pblocks, pb, NT * kThreads) + tid; };
  const size_t state = ((size_t)p.n * a.H + h) * N * a.P + col0 + wcol + l16;
  const bool from_front = outputs && (p.j > 0 || (p.parts > 1 && a.keep));
  const bool live = col0 + wcol < a.P;                   // (P is a multiple of 16)
  if (from_front) {
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = front(p.j)[k * kThreads];
  } else if (p.j == 0 && a.initial_state && live) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k][i] = a.initial_state[state + (size_t)(16 * k + 4 * g + i) * a.P];
  } else {
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (!outputs && p.j == 0 && a.keep)
#pragma unroll
    for (int k = 0; k < NT; ++k) front(0)[k * kThreads] = s[k];

  // ---- loads of a chunk into registers, and from there into LDS: 16 bytes each, two
  // of x a thread, UB of B and of C.
  constexpr int XV = 2 * W, kXRows = kThreads / XV, kRows = kThreads / NV, kUnits = kL * NV;
  constexpr int UB = (kUnits + kThreads - 1) / kThreads;
  static_assert(kXRows == kL / 2 && kThreads % NV == 0, "rows of a thread");
  static_assert(kRows % 8 == 0, "a row's mask is that of its first row XOR that of the rows between");
  u32x4 rx[2], rb[UB], rc[UB];
  // Byte offsets of a thread's rows from a chunk's first token (64 rows of at most
  // KDA_SSM_MAX_STRIDE elements: below 2^31). What is the same for all is kept in
  // scalars.
  const char* gx = (const char*)((const bf16_bits*)a.x + p.first * a.x_stride + (int64_t)h * a.P + col0);
  const char* gb = (const char*)((const bf16_bits*)a.b + p.first * a.b_stride + grp * N);
  const char* gc = (const char*)((const bf16_bits*)a.c + p.first * a.c_stride + grp * N);
  const uint32_t xs = 2 * (uint32_t)a.x_stride, bs = 2 * (uint32_t)a.b_stride, cs = 2 * (uint32_t)a.c_stride;
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  const Minus one = minus_one();
  // (columns behind the head's: the first ones again, nothing is made of them)
  const uint32_t xcol = col0 + 8 * (tid % XV) < a.P ? 16 * (tid % XV) : 0, bcol = 16 * (tid % NV);
  const uint32_t xoff = tid / XV * xs + xcol, boff = tid / NV * bs + bcol, coff = tid / NV * cs + bcol;
  // Of the last chunk of a segment, rows behind the end are read as its last row
  // (offsets grow with the row, so the smaller of two is the earlier row): their
  // step sizes are 0, so nothing is added by them, and no output is theirs.
  auto load = [&](int t0) __attribute__((always_inline)) {
    const uint32_t rows = min(p.count - t0, kL) - 1;
    const uint32_t x1 = fresh(xcol) + rows * xs, b1 = fresh(bcol) + rows * bs;
#pragma unroll
    for (int k = 0; k < 2; ++k) rx[k] = *(const u32x4*)(gx + min(xoff + k * kXRows * xs, x1));
#pragma unroll
    for (int k = 0; k < UB; ++k) rb[k] = *(const u32x4*)(gb + min(boff + k * kRows * bs, b1));
    gx += (int64_t)kL * xs;
    gb += (int64_t)kL * bs;
  };
  auto load_c = [&](int t0) __attribute__((always_inline)) {
    const uint32_t rows = min(p.count - t0, kL) - 1, c1 = fresh(bcol) + rows * cs;
#pragma unroll
    for (int k = 0; k < UB; ++k) rc[k] = *(const u32x4*)(gc + min(coff + k * kRows * cs, c1));
    gc += (int64_t)kL * cs;
  };
  const int xplace = tid / XV * kCols + (tid % XV ^ row_mask<kCols>(tid / XV % 16)) * 8;
  const int bplace = tid / NV * NP + channel_place<NP>(tid % NV, tid / NV % 16);
  // The chunk in front leaves its outputs in the place of its x, and the threads that
  // put x there write them out: whole rows, past the caches (so that they are not
  // still in them when the kernel ends).
  const int64_t yrow = 2 * (int64_t)a.H * a.P;
  char* gy = (char*)((bf16_bits*)a.y + ((size_t)p.first * a.H + h) * a.P + col0);
  const uint32_t yoff = tid / XV * (uint32_t)yrow + 16 * (tid % XV);
  auto write_out = [&](int t0) __attribute__((always_inline)) {
    const uint32_t t = fresh(threadIdx.x), at = fresh(yoff);
    if (col0 + 8 * (int)(t % XV) < a.P)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (t0 + (int)(t / XV) + k * kXRows < p.count)
          __builtin_nontemporal_store(*(const u32x4*)(sX + xplace + k * kXRows * kCols),
                                      (u32x4*)(gy + k * kXRows * yrow + at));
    gy += kL * yrow;
  };
  auto store = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2; ++k) *(u32x4*)(sX + xplace + k * kXRows * kCols) = rx[k];
    const int at = fresh(bplace);
#pragma unroll
    for (int k = 0; k < UB; ++k)
      if (kUnits % kThreads == 0 || tid + k * kThreads < kUnits) {
        store_channels(sB + k * kRows * NP, at ^ row_mask<NP>(k * kRows % 16) * 8, rb[k]);
        if (outputs) store_channels(sC + k * kRows * NP, at ^ row_mask<NP>(k * kRows % 16) * 8, rc[k]);
      }
  };
  if (N < NP && outputs && tid < kL)                     // the channels of a row of 32 that N = 16 leaves
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int at = tid * NP + (b ^ row_mask<NP>(tid % 16)) * 8 + 4;
      *(uint2*)(sB + at) = uint2{0u, 0u}, *(uint2*)(sC + at) = uint2{0u, 0u};
    }
  // A lane's places as it reads: row l16 and block g of a tile of M and of B or C; and
  // turned over, columns 4 (l16 % 4) of row 4 g + l16 / 4 of x (the wave's) and B.
  const int turned = 4 * g + l16 / 4, quad = l16 % 4;
  const int token_read = l16 * kL + (g ^ row_mask<kL>(l16)) * 8;
  const int channel_read = l16 * NP + (g ^ row_mask<NP>(l16)) * 8;
  const int x_turned = turned * kCols + (2 * wave + quad / 2 ^ row_mask<kCols>(turned)) * 8 + 4 * (quad & 1);
  const int ywrite = l16 * kCols + (2 * wave + g / 2 ^ row_mask<kCols>(l16)) * 8 + 4 * (g & 1);
  const int b_turned = turned * NP + (quad ^ row_mask<NP>(turned)) * 8;

  // Wave w, lane t: what becomes of dt in the w-th of the next four chunks.
  float rdt = 0.f;
  double sum = 0.0;                                      // of the segment's d a, in the four waves' parts
  auto load_dt = [&](int t0) __attribute__((always_inline)) {
    const int t = t0 + fresh(threadIdx.x);                       // (kL * wave + lane)
    rdt = uwave < 4 && t < p.count ? a.dt[(size_t)(p.first + t) * a.H + h] : 0.f;
  };
  auto decays = [&](int t0) __attribute__((always_inline)) {
    if (uwave >= 4 || t0 + kL * uwave >= p.count) return;
    const uint32_t t = fresh(threadIdx.x);
    const bool on = t0 + (int)t < p.count;
    const float d = on ? step_size(rdt, bias, a.softplus) : 0.f;
    const double end = make_decays<kL>(on, d, av, t % kWave, dec + uwave);
    if (!outputs) sum += end;
  };

  // A chunk that grows: the recurrence, as a step computes it. Outputs go to the place of
  // x, which only this wave reads. The state rests in scratch memory, and the loads of it
  // end here: in registers, or waited for behind this path, it costs the others 2 to 7 %.
  auto by_tokens = [&](const Decays<kL>& q, int count) __attribute__((always_inline)) {
    f32x4 states[NT];
    in_memory(states);
#pragma unroll
    for (int k = 0; k < NT; ++k) states[k] = s[k];
    const int ft = fresh(threadIdx.x), fg = ft / 16 % 4, c8 = 2 * wave + ft % 16 / 8;
#pragma unroll 1
    for (int t = 0; t < count; ++t) {
      bf16_bits* const px = sX + t * kCols + (c8 ^ row_mask<kCols>(t % 16)) * 8 + ft % 8;
      const int at = t * NP, mask = row_mask<NP>(t % 16);
      const float x = bf16_to_f32(*px), d = uniform(q.d[t]), da = d * av, f = expf(da > kMostGrowth ? kMostGrowth : da);
      float o = 0.f;
#pragma unroll 1
      for (int k = 0; k < NT; ++k) {
        const int place = at + ((4 * (k / 2) + fg) ^ mask) * 8 + 4 * (k & 1);
        f32x4 v = states[k];
        if (da > kMostGrowth) v = grown(v, da);
        v = f * v + d * from_bf16x4(*(const bf16x4*)(sB + place)) * x;
        states[k] = v;
        if (outputs) {
          const f32x4 r = from_bf16x4(*(const bf16x4*)(sC + place)) * v;
          o += (r[0] + r[1]) + (r[2] + r[3]);
        }
      }
      if (outputs) {
        o += __shfl_xor(o, 16);
        o += __shfl_xor(o, 32);
        if (a.skip) o += skip * x;
        if (fg == 0) *px = f32_to_bf16_bits(o);
      }
    }
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = fresh(states[k]);
  };

  load_dt(0);
  if (p.count > 0) {
    load(0);
    if (outputs) load_c(0);
  }
  // Chunks from token t0 on, up to one that grows.
  auto chunks = [&](int t0) __attribute__((always_inline)) {
#pragma unroll 1
    for (; t0 < p.count; t0 += kL) {
      const Decays<kL>& q = dec[t0 / kL & 3];
      if ((t0 / kL & 3) == 0) {
        decays(t0);
        load_dt(t0 + 4 * kL);
      }
      if (outputs && t0 > 0) write_out(t0 - kL);
      store();
      lds_barrier();
      if (t0 + kL < p.count) load(t0 + kL);
      if (__builtin_expect(__builtin_amdgcn_readfirstlane(q.grows), 0)) break;
      f32x4 y[4];
      if (outputs) {
        // ---- M, transposed (a lane: one t, 4 s each), in tiles of 16 t by 16 s: the
        // ten up to the diagonal and two of zeros, shared out over the waves
        constexpr int kTiles = 12, kPer = (kTiles + W - 1) / W;
        const int cr = fresh(channel_read), mr = fresh(token_read);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int id = uwave + k * W;
          // tiles (tt, u) by id: 0 .. 3 (3, u), 4 .. 6 (2, u), 7 (1, 0), 8 (1, 1), 9 (0, 0), 10 (0, 1), 11 (2, 3)
          const int tt = id < 4 ? 3 : id < 7 ? 2 : id < 9 ? 1 : id < 11 ? 0 : 2;
          const int u = id < 4 ? id : id < 7 ? id - 4 : id < 9 ? id - 7 : id < 11 ? id - 9 : 3;
          f32x4 x = {0.f, 0.f, 0.f, 0.f};
          if (id < 10) {
            const int t = 16 * tt + l16;
            bf16x8 b[KS], c[KS];
#pragma unroll
            for (int v = 0; v < KS; ++v) {
              b[v] = *(const bf16x8*)(sB + (cr ^ 32 * v) + 16 * u * NP);
              c[v] = *(const bf16x8*)(sC + (cr ^ 32 * v) + 16 * tt * NP);
            }
#pragma unroll
            for (int v = 0; v < KS; ++v) x = mfma32(b[v], c[v], x);
            const float thi = q.hi[t], tlo = q.lo[t];
            const f32x4 shi = *(const f32x4*)&q.hi[16 * u + 4 * g], slo = *(const f32x4*)&q.lo[16 * u + 4 * g],
                        sd = *(const f32x4*)&q.d[16 * u + 4 * g];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] *= __builtin_amdgcn_exp2f((thi - shi[i]) + (tlo - slo[i])) * sd[i];
            if (u == tt) {
              const int at = fresh(l16) - 4 * g;                // the diagonal's place among the lane's 4
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float v = i == at ? x[i] + skip : x[i];
                x[i] = i <= at ? v : 0.f;
              }
            }
          }
          bf16x4 mh, mm, ml;
          split3(x, mh, mm, ml, one);
          const int at = (mr ^ 32 * (u / 2)) + 16 * tt * kL + 4 * (u & 1);
          if (id < kTiles) {
            *(bf16x4*)(sM[0] + at) = mh;
            *(bf16x4*)(sM[1] + at) = mm;
            *(bf16x4*)(sM[2] + at) = ml;
          }
        }
        // ---- y, transposed (a lane: one t, 4 columns): the state's part first
        // (it needs nothing of M, which the other waves finish meanwhile)
        const int hr = fresh(channel_read);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) y[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < KS; ++v) {
          bf16x4 h0, m0, l0, h1 = {}, m1 = {}, l1 = {};
          split3(s[2 * v], h0, m0, l0, one);
          if constexpr (NT > 1) split3(s[2 * v + 1], h1, m1, l1, one);
          const bf16x8 sh = cat(h0, h1), sm = cat(m0, m1), sl = cat(l0, l1);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
            const bf16x8 c = *(const bf16x8*)(sC + (hr ^ 32 * v) + 16 * tt * NP);
            y[tt] = mfma32(sl, c, y[tt]);
            y[tt] = mfma32(sm, c, y[tt]);
            y[tt] = mfma32(sh, c, y[tt]);
          }
        }
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) y[tt] *= q.e[16 * tt + l16];
        lds_barrier();
      }
      // ---- x of the wave's columns: operands of both products
      auto x_operand = [&](int v) __attribute__((always_inline)) {
        const bf16_bits* at = sX + x_turned + 32 * v * kCols;
        return cat(read_turned(at), read_turned(at + 16 * kCols));
      };
      bf16x8 xo[2] = {x_operand(0), x_operand(1)};
      if (outputs) {
        // A value that is not finite would reach earlier tokens through M's zeros:
        // it is taken out here, and its column made NaN from its token on.
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 most = {0, 0};
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const u32x4 bits = __builtin_bit_cast(u32x4, xo[v]) & 0x7fff7fffu;
#pragma unroll
          for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, (uint32_t)bits[i]));
        }
        const bool bad = most[0] >= 0x7f80 || most[1] >= 0x7f80;
        const bool any_bad = __any(bad);
        int from = kL;
        if (any_bad) {
          const int fg = fresh(threadIdx.x) / 16 % 4;
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (!((float)xo[v][i] * 0.f == 0.f)) {
                xo[v][i] = (__bf16)0.f;
                from = min(from, 32 * v + 16 * (i / 4) + 4 * fg + i % 4);
              }
          from = min(from, __builtin_amdgcn_ds_bpermute(4 * (fresh(threadIdx.x) ^ 16), from));
          from = min(from, __builtin_amdgcn_ds_bpermute(4 * (fresh(threadIdx.x) ^ 32), from));
        }
        const int mr = fresh(token_read);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int v = 0; v <= tt / 2; ++v) {
            const int at = (mr ^ 32 * v) + 16 * tt * kL;
#pragma unroll
            for (int k = 2; k >= 0; --k) y[tt] = mfma32(xo[v], *(const bf16x8*)(sM[k] + at), y[tt]);
          }
        if (any_bad) {
          const uint32_t ft = fresh(threadIdx.x);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int first = __builtin_amdgcn_ds_bpermute(4 * (ft / 16 % 4 * 4 + i), from);
#pragma unroll
            for (int tt = 0; tt < 4; ++tt)
              if (16 * tt + (int)(ft % 16) >= first) y[tt][i] = __builtin_nanf("");
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) xo[v] = x_operand(v);
        }
        // (x of the wave's columns is in registers, and no other wave reads it)
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) *(bf16x4*)(sX + ywrite + 16 * tt * kCols) = to_bf16x4(y[tt]);
        if (t0 + kL < p.count) load_c(t0 + kL);            // (late: the registers are needed until here)
      }
      // ---- the state behind the chunk
      const float total = q.total;
      const int br = fresh(b_turned);
#pragma unroll
      for (int k = 0; k < NT; ++k) s[k] *= total;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        bf16x4 h0, m0, l0, h1, m1, l1;
        split3(from_bf16x4(lo_half(xo[v])) * *(const f32x4*)&q.w[32 * v + 4 * g], h0, m0, l0, one);
        split3(from_bf16x4(hi_half(xo[v])) * *(const f32x4*)&q.w[32 * v + 16 + 4 * g], h1, m1, l1, one);
        const bf16x8 xh = cat(h0, h1), xm = cat(m0, m1), xl = cat(l0, l1);
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          const bf16_bits* at = sB + (br ^ 32 * (k / 2)) + 4 * (k & 1) + 32 * v * NP;
          const bf16x8 b = cat(read_turned(at), read_turned(at + 16 * NP));
          s[k] = mfma32(b, xl, s[k]);
          s[k] = mfma32(b, xm, s[k]);
          s[k] = mfma32(b, xh, s[k]);
        }
      }
      lds_barrier();                                       // the chunk is used
    }
    return t0;
  };
  // (a loop of its own, which keeps its registers)
  for (int t0 = 0; (t0 = chunks(t0)) < p.count; t0 += kL) {
    by_tokens(dec[t0 / kL & 3], min(p.count - t0, kL));
    if (outputs && t0 + kL < p.count) load_c(t0 + kL);
    lds_barrier();
  }
  if (outputs && p.count > 0) write_out((p.count - 1) / kL * kL);

  if (!outputs) {
#pragma unroll
    for (int k = 0; k < NT; ++k) front(p.j + 1)[k * kThreads] = s[k];
    if (pb == 0) {
      __shared__ double part[4];
      if (lane == 0 && wave < 4) part[wave] = sum;
      __syncthreads();
      if (tid == 0) a.sums[entry_of(a, p, h, p.j)] = part[0] + part[1] + part[2] + part[3];
    }
  } else if (last && a.final_state && live) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.final_state[state + (size_t)(16 * k + 4 * g + i) * a.P] = s[k][i];
  }
}

// ---- fp32: chunks of 32 tokens on the matrix cores --------------------------------------
//
// The same, with products of fp32 (16 x 16 x 4): no factor is split. 64 columns a
// workgroup, 16 a wave. As operand a lane holds 4 values along the sum, each for
// one of four products: the accumulators of a tile are that operand as they are
// (rows 16 k + 4 g + i, i the product), and 4 channels or tokens are one read.
// Layouts as above, with blocks of 4 fp32. 8192 tokens of 32 heads 128 x 128: 351 us,
// of which the products take 139 at the rate of a large fp32 product (154 TFLOP/s) in
// the launch with outputs, and 2/5 of that again in the one for states; nine sequences
// of 3001 tokens, 6 heads 32 x 48: 20 us, three chunks after each other in each pass.
// By tokens, a state in registers: 830 and 62 us.
constexpr int kL32 = 32;

__device__ __forceinline__ f32x4 mfma4(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

template <int N, bool outputs>
__global__ __launch_bounds__(256, waves_of(N, 4, outputs)) void ssm_chunk32_kernel(SsmParams a) {
  constexpr int kThreads = 256, kCols = 64, L = kL32, NT = N / 16, NV = N / 4;
  const int pblocks = (a.P + kCols - 1) / kCols;
  const int id = numbered(shared_groups(a.H / a.G, pblocks));
  const int pb = id % pblocks, h = id / pblocks % a.H;
  Part p;
  if (!find_part(a.seqs, a.len, id / pblocks / a.H, p)) return;
  const bool last = p.j == p.parts - 1;
  if (!outputs && last) return;
  const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, g = lane / 16, l16 = lane % 16;
  const int wcol = wave * 16, col0 = pb * kCols, grp = h / (a.H / a.G);
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  const float av = a.a[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, skip = a.skip ? a.skip[h] : 0.f;

  constexpr int kB = L * N, kM = L * L;
  __shared__ __attribute__((aligned(16))) float sC[L * N], sBM[kB > kM ? kB : kM], sBT[N * L], sXT[kCols * L];
  __shared__ Decays<L> dec[8];
  float *sB = sBM, *sM = sBM;                            // (M overwrites B once it is used)

  f32x4 s[NT];
  auto front = [&](int j) { return front_of(a, p, h, j, pblocks, pb, NT * kThreads) + tid; };
  const size_t state = ((size_t)p.n * a.H + h) * N * a.P + col0 + wcol + l16;
  const bool live = col0 + wcol < a.P;                   // (P is a multiple of 16)
  if (outputs && (p.j > 0 || (p.parts > 1 && a.keep))) {
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = front(p.j)[k * kThreads];
  } else if (p.j == 0 && a.initial_state && live) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[k][i] = a.initial_state[state + (size_t)(16 * k + 4 * g + i) * a.P];
  } else {
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (!outputs && p.j == 0 && a.keep)
#pragma unroll
    for (int k = 0; k < NT; ++k) front(0)[k * kThreads] = s[k];

  // Runs of 4 tokens by 4 columns of x (128) and B (8 N / 4), rows of C.
  constexpr int kXRuns = 16 * 8, kRuns = kXRuns + NV * 8, UR = (kRuns + kThreads - 1) / kThreads;
  constexpr int kCUnits = L * NV, UC = (kCUnits + kThreads - 1) / kThreads;
  f32x4 rr[UR][4], rc[UC];
  const char* gx = (const char*)((const float*)a.x + p.first * a.x_stride + (int64_t)h * a.P + col0);
  const char* gb = (const char*)((const float*)a.b + p.first * a.b_stride + grp * N);
  const char* gc = (const char*)((const float*)a.c + p.first * a.c_stride + grp * N);
  const int64_t xs = 4 * a.x_stride, bs = 4 * a.b_stride, cs = 4 * a.c_stride;
  auto of_x = [&](int k) { return uwave * kWave + k * kThreads < kXRuns; };
  // (run i: columns 4 (i % 4 + 4 (i / 32)), tokens 4 (i / 4 % 8))
  auto run_col = [&](int k, uint32_t t) -> int {
    const uint32_t i = t + k * kThreads - (of_x(k) ? 0 : kXRuns);
    return i % 4 + 4 * (i / 32);
  };
  auto run_tok = [&](uint32_t t) -> int { return t / 4 % 8; };
  uint32_t first[UR], off[UR];
#pragma unroll
  for (int k = 0; k < UR; ++k) {
    const int cv = run_col(k, tid);
    first[k] = (of_x(k) ? col0 + 4 * cv < a.P : tid + k * kThreads < kRuns) ? 16 * cv : 0;
    off[k] = 4 * run_tok(tid) * (uint32_t)(of_x(k) ? xs : bs) + first[k];
  }
  const uint32_t coff = tid / NV * (uint32_t)cs + tid % NV * 16;
  auto load = [&](int t0) __attribute__((always_inline)) {
    const uint32_t rows = min(p.count - t0, L) - 1;
#pragma unroll
    for (int k = 0; k < UR; ++k) {
      const char* base = of_x(k) ? gx : gb;
      const uint32_t step = (uint32_t)(of_x(k) ? xs : bs), most = first[k] + rows * step;
#pragma unroll
      for (int r = 0; r < 4; ++r) rr[k][r] = *(const f32x4*)(base + min(off[k] + r * step, most));
    }
    if (outputs) {
      const uint32_t most = tid % NV * 16 + rows * (uint32_t)cs;
#pragma unroll
      for (int k = 0; k < UC; ++k)
        rc[k] = *(const f32x4*)(gc + min(coff + k * (kThreads / NV) * (uint32_t)cs, most));
    }
    gx += L * xs;
    gb += L * bs;
    gc += L * cs;
  };
  // (masks of rows by their bytes: a row of 2 N bf16 is one of N fp32)
  auto store = [&]() __attribute__((always_inline)) {
    const uint32_t t = fresh(threadIdx.x);
#pragma unroll
    for (int k = 0; k < UR; ++k) {
      if (kRuns % kThreads != 0 && t + k * kThreads >= kRuns) continue;
      const int cv = run_col(k, t), sr = run_tok(t);
      float* dst = of_x(k) ? sXT : sBT;
#pragma unroll
      for (int c = 0; c < 4; ++c) {                      // column 4 cv + c: row 4 (cv & 3) + c of its tile
        const int l = 4 * (cv & 3) + c;
        *(f32x4*)(dst + (16 * (cv / 4) + (l ^ (cv / 4 & 1))) * L + (sr ^ l >> 1) * 4) =
            f32x4{rr[k][0][c], rr[k][1][c], rr[k][2][c], rr[k][3][c]};
      }
      if (outputs && !of_x(k))
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *(f32x4*)(sB + (4 * sr + r) * N + (cv ^ row_mask<2 * N>(4 * (sr & 3) + r)) * 4) = rr[k][r];
    }
    if (outputs)
#pragma unroll
      for (int k = 0; k < UC; ++k) {
        const int row = t / NV + k * (kThreads / NV);
        if (kCUnits % kThreads == 0 || t + k * kThreads < kCUnits)
          *(f32x4*)(sC + row * N + (t % NV ^ row_mask<2 * N>(row % 16)) * 4) = rc[k];
      }
  };
  const int token_read[2] = {l16 * L + (g ^ l16 >> 1) * 4, (l16 ^ 1) * L + (g ^ l16 >> 1) * 4};
  const int channel_read = l16 * N + (g ^ row_mask<2 * N>(l16)) * 4;

  // Wave w, lane t: what becomes of dt in the 2 w-th and next of the next eight chunks.
  float rdt = 0.f;
  double sum = 0.0;
  auto load_dt = [&](int t0) __attribute__((always_inline)) {
    const int t = t0 + tid;
    rdt = t < p.count ? a.dt[(size_t)(p.first + t) * a.H + h] : 0.f;
  };
  auto decays = [&](int t0) __attribute__((always_inline)) {
    if (t0 + 2 * L * uwave >= p.count) return;
    const uint32_t t = fresh(threadIdx.x);
    const bool on = t0 + (int)t < p.count;
    const float d = on ? step_size(rdt, bias, a.softplus) : 0.f;
    const double end = make_decays<L>(on, d, av, t % kWave, dec + 2 * uwave);
    if (!outputs) sum += end;                            // (a lane: of its half of the wave)
  };

  const int64_t yrow = 4 * (int64_t)a.H * a.P;
  char* gy = (char*)((float*)a.y + ((size_t)p.first * a.H + h) * a.P + col0);
  auto by_tokens = [&](const Decays<L>& q, int count) __attribute__((always_inline)) {
    f32x4 states[NT];
    in_memory(states);
#pragma unroll
    for (int k = 0; k < NT; ++k) states[k] = s[k];
    const int ft = fresh(threadIdx.x), fg = ft / 16 % 4, fl = ft % 16;
#pragma unroll 1
    for (int t = 0; t < count; ++t) {
      // (token t of row l of a tile: its four of tokens is at t / 4 ^ l / 2)
      auto place = [&](int tile, int l) { return (16 * tile + (l ^ (tile & 1))) * L + (t / 4 ^ l >> 1) * 4 + t % 4; };
      const float x = sXT[place(uwave, fl)], d = uniform(q.d[t]), da = d * av, f = expf(da > kMostGrowth ? kMostGrowth : da);
      float o = 0.f;
#pragma unroll 1
      for (int k = 0; k < NT; ++k) {
        f32x4 b, v = states[k];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = sBT[place(k, 4 * fg + i)];
        if (da > kMostGrowth) v = grown(v, da);
        v = f * v + d * b * x;
        states[k] = v;
        if (outputs) {
          const f32x4 r = *(const f32x4*)(sC + t * N + ((4 * k + fg) ^ row_mask<2 * N>(t % 16)) * 4) * v;
          o += (r[0] + r[1]) + (r[2] + r[3]);
        }
      }
      if (outputs) {
        o += __shfl_xor(o, 16);
        o += __shfl_xor(o, 32);
        if (a.skip) o += skip * x;
        if (live && fg == 0) *(float*)(gy + t * yrow + 4 * (16 * uwave + fl)) = o;
      }
    }
    gy += L * yrow;
#pragma unroll
    for (int k = 0; k < NT; ++k) s[k] = fresh(states[k]);
  };

  load_dt(0);
  if (p.count > 0) load(0);
  auto chunks = [&](int t0) __attribute__((always_inline)) {
#pragma unroll 1
    for (; t0 < p.count; t0 += L) {
      const Decays<L>& q = dec[t0 / L & 7];
      if ((t0 / L & 7) == 0) {
        decays(t0);
        load_dt(t0 + 8 * L);
      }
      store();
      lds_barrier();
      if (t0 + L < p.count) load(t0 + L);
      if (__builtin_expect(__builtin_amdgcn_readfirstlane(q.grows), 0)) break;
      if (outputs) {
        // ---- M: tiles (tt, u) = (0, 0), (1, 0), (1, 1), a wave each
        const int tt = uwave > 0, u = uwave == 2;
        f32x4 m = {0.f, 0.f, 0.f, 0.f};
        const int cr = fresh(channel_read);
        if (uwave < 3) {
          const int t = 16 * tt + l16;
#pragma unroll
          for (int k = 0; k < NT; ++k)
            m = mfma4(*(const f32x4*)(sB + (cr ^ 16 * k) + 16 * u * N), *(const f32x4*)(sC + (cr ^ 16 * k) + 16 * tt * N), m);
          const float thi = q.hi[t], tlo = q.lo[t];
          const f32x4 shi = *(const f32x4*)&q.hi[16 * u + 4 * g], slo = *(const f32x4*)&q.lo[16 * u + 4 * g],
                      sd = *(const f32x4*)&q.d[16 * u + 4 * g];
#pragma unroll
          for (int i = 0; i < 4; ++i) m[i] *= __builtin_amdgcn_exp2f((thi - shi[i]) + (tlo - slo[i])) * sd[i];
          if (u == tt) {
            const int at = fresh(l16) - 4 * g;             // the diagonal's place among the lane's 4
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float v = i == at ? m[i] + skip : m[i];
              m[i] = i <= at ? v : 0.f;
            }
          }
        }
        lds_barrier();                                     // B is used
        if (uwave < 3) *(f32x4*)(sM + 16 * tt * L + (token_read[0] ^ 16 * u)) = m;
        lds_barrier();
      }
      auto x_operand = [&](int u) __attribute__((always_inline)) {
        return *(const f32x4*)(sXT + (fresh(token_read[uwave & 1]) ^ 16 * u) + uwave * 16 * L);
      };
      f32x4 xo[2] = {x_operand(0), x_operand(1)};
      if (outputs) {
        f32x4 y[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int cr = fresh(channel_read);
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int tt = 0; tt < 2; ++tt) y[tt] = mfma4(s[k], *(const f32x4*)(sC + (cr ^ 16 * k) + 16 * tt * N), y[tt]);
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) y[tt] *= q.e[16 * tt + l16];
        // (values that are not finite: as above)
        bool bad = false;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) bad |= !(fabsf(xo[u][i]) < __builtin_inff());
        const bool any_bad = __any(bad);
        int from = L;
        if (any_bad) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(fabsf(xo[u][i]) < __builtin_inff())) {
                xo[u][i] = 0.f;
                from = min(from, 16 * u + 4 * g + i);
              }
          from = min(from, __shfl_xor(from, 16));
          from = min(from, __shfl_xor(from, 32));
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
          for (int u = 0; u <= tt; ++u)
            y[tt] = mfma4(xo[u], *(const f32x4*)(sM + 16 * tt * L + (token_read[0] ^ 16 * u)), y[tt]);
        if (any_bad) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int first_bad = __shfl(from, 4 * g + i);
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
              if (16 * tt + l16 >= first_bad) y[tt][i] = __builtin_nanf("");
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) xo[u] = x_operand(u);
        }
        if (live) {
          const int left = p.count - t0 - l16;
          const uint32_t yoff = l16 * (uint32_t)yrow + 4 * (16 * uwave + 4 * g);
#pragma unroll
          for (int tt = 0; tt < 2; ++tt)
            if (16 * tt < left) *(f32x4*)(gy + 16 * tt * yrow + yoff) = y[tt];
        }
        gy += L * yrow;
      }
      const float total = q.total;
#pragma unroll
      for (int k = 0; k < NT; ++k) s[k] *= total;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 xw = xo[u] * *(const f32x4*)&q.w[16 * u + 4 * g];
#pragma unroll
        for (int k = 0; k < NT; ++k)
          s[k] = mfma4(*(const f32x4*)(sBT + (token_read[k & 1] ^ 16 * u) + 16 * k * L), xw, s[k]);
      }
      lds_barrier();                                       // the chunk is used
    }
    return t0;
  };
  for (int t0 = 0; (t0 = chunks(t0)) < p.count; t0 += L) {
    by_tokens(dec[t0 / L & 7], min(p.count - t0, L));
    lds_barrier();
  }

  if (!outputs) {
#pragma unroll
    for (int k = 0; k < NT; ++k) front(p.j + 1)[k * kThreads] = s[k];
    if (pb == 0) {
      __shared__ double part[8];
      if (lane % L == 0) part[tid / L] = sum;
      __syncthreads();
      if (tid == 0) {
        for (int i = 1; i < 8; ++i) sum += part[i];
        a.sums[entry_of(a, p, h, p.j)] = sum;
      }
    }
  } else if (last && a.final_state && live) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) a.final_state[state + (size_t)(16 * k + 4 * g + i) * a.P] = s[k][i];
  }
}

// The states in front of the segments of one sequence (a block per 256 vectors of
// them and per multiple of len, where at most one sequence of several segments
// starts). vecs: vectors of a head's state. Bound by HBM: 16 segments of 32 heads
// 128 x 128 are 64 MB read and written in 13 us, 4.9 TB/s.
__global__ __launch_bounds__(kThreads) void ssm_front_kernel(SsmParams a, int blocks, int vecs) {
  const int b = blockIdx.x % blocks, h = blockIdx.x / blocks % a.H, at = blockIdx.x / blocks / a.H;
  Part p;
  int end;
  p.n = last_sequence(a.seqs, a.len, 0, at, p.start, end);   // the last that starts before (at + 1) len
  p.length = end - p.start;
  const int i = b * kThreads + threadIdx.x;
  if (p.start / a.len != at || p.length <= 2 * a.len || i >= vecs) return;
  const int parts = (p.length - 1) / a.len + 1;
  const size_t step = (size_t)a.H * vecs;
  f32x4* v = (f32x4*)a.ends + entry_of(a, p, h, 1) * vecs + i;
  f32x4 s = *v;
  constexpr int U = 4;                // segments whose states are on their way at once
  for (int j = 1; j < parts - 1; j += U) {
    const int m = min(U, parts - 1 - j);
    f32x4 e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) e[u] = v[(size_t)(min(u, m - 1) + 1) * step];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < m) {
        double sum = a.sums[entry_of(a, p, h, j + u)];
        if (sum > kMostGrowth) s = grown(s, (float)sum), sum = kMostGrowth;
        s = __builtin_amdgcn_exp2f((float)(sum * 1.4426950408889634)) * s + e[u];
        v[(size_t)(u + 1) * step] = s;
      }
    v += (size_t)m * step;
  }
}

// One token: the state read and written once, a float4 of columns per thread
// and as many rows at a time as the workgroup has threads for (the rest idles
// where P / 4 does not divide it). A workgroup takes the whole head, or where
// that leaves compute units without one, a part of its columns. Bound by HBM: 256
// sequences of 32 heads 128 x 128, 1.08 GB: 207 us, 5.2 TB/s.
template <typename T>
__global__ __launch_bounds__(kThreads) void ssm_step_kernel(SsmParams a, int N, int split) {
  const int part_id = blockIdx.x % split, h = blockIdx.x / split % a.H, n = blockIdx.x / split / a.H;
  const int cols = a.P / split, vecs = cols / 4, groups = kThreads / vecs;
  const int tid = threadIdx.x, cv = tid % vecs, rg = tid / vecs, col = part_id * cols + cv * 4;
  const int grp = h / (a.H / a.G);
  __shared__ float sb[256], sc[256];
  __shared__ f32x4 part[kThreads];
  const bool on = rg < groups;
  float* S = a.final_state + ((size_t)n * a.H + h) * N * a.P + col;
  // (the state's first rows are on their way while d and B are made)
  constexpr int U = 8;
  f32x4 s[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (on) s[u] = *(const f32x4*)(S + (size_t)min(rg + u * groups, N - 1) * a.P);
  const float d = step_size(a.dt[(size_t)n * a.H + h], a.dt_bias ? a.dt_bias[h] : 0.f, a.softplus);
  const float da = d * a.a[h], f = expf(da > kMostGrowth ? kMostGrowth : da);
  if (tid < N) {
    sb[tid] = d * Elem<T>::load((const T*)a.b + n * a.b_stride + grp * N + tid);
    sc[tid] = Elem<T>::load((const T*)a.c + n * a.c_stride + grp * N + tid);
  }
  float xv[4];
  load_vec<T, 4>((const T*)a.x + n * a.x_stride + (int64_t)h * a.P + col, xv);
  const f32x4 x = {xv[0], xv[1], xv[2], xv[3]};
  lds_barrier();
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  auto rows = [&](auto grows) __attribute__((always_inline)) {
    for (int r0 = rg; on && r0 < N; r0 += U * groups) {
      if (r0 != rg)
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] = *(const f32x4*)(S + (size_t)min(r0 + u * groups, N - 1) * a.P);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * groups;
        if (r < N) {
          if constexpr (decltype(grows)::value) s[u] = grown(s[u], da);
          s[u] = f * s[u] + sb[r] * x;
          o += sc[r] * s[u];
          __builtin_nontemporal_store(s[u], (f32x4*)(S + (size_t)r * a.P));
        }
      }
    }
  };
  if (__builtin_expect(uniform(da) > kMostGrowth, 0)) rows(std::true_type{});
  else rows(std::false_type{});
  // sums over the groups of rows, halved until one is left
  for (int m = groups; m > 1;) {
    part[tid] = o;
    lds_barrier();
    const int half = (m + 1) / 2;
    if (rg + half < m) o += part[tid + half * vecs];
    m = half;
    lds_barrier();
  }
  if (tid < vecs) {
    if (a.skip) o += a.skip[h] * x;
    const float out[4] = {o[0], o[1], o[2], o[3]};
    store_vec<T, 4>((T*)a.y + ((size_t)n * a.H + h) * a.P + col, out);
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
  p.keep = a.initial_state && a.initial_state == a.final_state;
  p.ends = nullptr; p.sums = nullptr;
  return p;
}

int64_t entries(const Packed& s, int len) { return len < s.T ? 2 * (int64_t)(s.T / len) : 0; }
size_t end_bytes(int H, int N, int P, const Split& sp) { return (size_t)H * column_blocks(sp, P) * sp.columns * N * 4; }

// Workgroups: whole rounds of the dies (the last ones have no segment).
int64_t launch_groups(const SsmArgs& a, const Split& sp) {
  const int64_t blocks = column_blocks(sp, a.P), round = kDies * shared_groups(a.H / a.G, blocks);
  const int64_t groups = part_slots(a.seqs, segment_len(a.seqs, a.H, a.N, a.P, sp)) * a.H * blocks;
  return (groups + round - 1) / round * round;
}

// All launches of a scan by a kernel (for states alone, and with outputs).
template <typename K>
hipError_t launch_passes(K states, K outputs, const SsmArgs& a, const Split& sp, int threads) {
  const int len = segment_len(a.seqs, a.H, a.N, a.P, sp);
  SsmParams p = params_of(a, len);
  const int64_t e = entries(a.seqs, len);
  p.ends = (float*)a.workspace;
  p.sums = (double*)((char*)a.workspace + e * end_bytes(a.H, a.N, a.P, sp));
  const unsigned groups = (unsigned)launch_groups(a, sp);
  if (e > 0) {
    hipLaunchKernelGGL(states, dim3(groups), dim3(threads), 0, a.stream, p);
    const int vecs = column_blocks(sp, a.P) * sp.columns * a.N / 4, blocks = (vecs + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(ssm_front_kernel, dim3((unsigned)(e / 2 * a.H * blocks)), dim3(kThreads), 0, a.stream, p, blocks,
                       vecs);
  }
  hipLaunchKernelGGL(outputs, dim3(groups), dim3(threads), 0, a.stream, p);
  return hipGetLastError();
}
template <int N>
hipError_t launch_n(const SsmArgs& a) {
  const Split sp = split_of(a.bf16, a.N, a.P);
  if (!a.bf16) return launch_passes(ssm_chunk32_kernel<N, false>, ssm_chunk32_kernel<N, true>, a, sp, 4 * sp.columns);
  if (a.P <= 64) return launch_passes(ssm_chunk_kernel<N, 4, false>, ssm_chunk_kernel<N, 4, true>, a, sp, 4 * sp.columns);
  return launch_passes(ssm_chunk_kernel<N, 8, false>, ssm_chunk_kernel<N, 8, true>, a, sp, 4 * sp.columns);
}

size_t workspace_of(int32_t T, int32_t H, int32_t N, int32_t P, const Split& sp) {
  const size_t by_target = (size_t)sp.target * ((size_t)sp.columns * N * 4 + 8);
  const size_t by_length = (size_t)(T / (2 * sp.chunk)) * (end_bytes(H, N, P, sp) + (size_t)H * 8);
  if (T <= sp.whole) return 0;
  return 2 * (by_target < by_length ? by_target : by_length);
}

}  // namespace

int64_t ssm_threads(const SsmArgs& a) {
  const Split sp = split_of(a.bf16, a.N, a.P);
  return launch_groups(a, sp) * 4 * sp.columns;
}

// At most 2 target / (H column blocks) entries, and at most two per 2
// chunks: both grow with the sizes. Any type, and heads narrow or wide: the
// largest.
size_t ssm_workspace(int32_t num_seqs, int32_t T, int32_t H, int32_t N, int32_t P) {
  (void)num_seqs;
  size_t most = 0;
  for (const Kind k : {kF32, kNarrow, kWide}) {
    if (k == kWide && P <= 64) continue;
    const size_t w = workspace_of(T, H, N, P, split_of(k, N));
    most = w > most ? w : most;
  }
  return most;
}

hipError_t launch_ssm(const SsmArgs& a) {
  switch (a.N) {
    case 16: return launch_n<16>(a);
    case 32: return launch_n<32>(a);
    case 64: return launch_n<64>(a);
    case 128: return launch_n<128>(a);
    default: return launch_n<256>(a);
  }
}

hipError_t launch_ssm_step(const SsmArgs& a) {
  SsmParams p = params_of(a, 1);
  const int64_t heads = (int64_t)a.seqs.num_seqs * a.H;
  // Halves of the columns until there are two workgroups a compute unit: 32 heads of
  // 128 x 128 whole 5.4 us, in quarters 4.3; of 8 sequences whole 9.6, in halves 8.8, in
  // quarters 11.2. Of at least 32 columns, a row's part a whole line: in parts of 16
  // three sequences take 9.0 us, in parts of 32 5.3.
  int split = 1;
  while (heads * split < 512 && a.P / split % 64 == 0) split *= 2;
  const dim3 grid((unsigned)(heads * split));
  if (a.bf16) hipLaunchKernelGGL(ssm_step_kernel<bf16_bits>, grid, dim3(kThreads), 0, a.stream, p, a.N, split);
  else hipLaunchKernelGGL(ssm_step_kernel<float>, grid, dim3(kThreads), 0, a.stream, p, a.N, split);
  return hipGetLastError();
}

}  // namespace kda
