// Verification of drafted tokens by rejection sampling on gfx950.
//
// At node `cur` with target row p and draft row q, after rejecting children
// 1 .. m the residual is r = max(p - C q, 0), C the sum of the masses so far:
// subtracting one more multiple of q from a row that is already clamped at 0
// gives the same as subtracting the total at once, so one number per node
// replaces a row of V. Every test needs p and q at one token only; a whole row
// is summed only for the mass after a rejection that another child follows,
// and for the draw of the next token.
//
// All sums are fp64: a token is chosen where a running sum of up to V values
// passes a threshold, and in fp32 the sum's rounding would be as wide as many
// tokens. Bound by the bytes of the rows p and q of the last node: 256 sequences
// and 131072 tokens of fp32 50 us, 5.4 TB/s.
//
// Three steps: the walk down the tree, the partial sums of the last node's r
// over chunks of the vocabulary, and the choice of the token inside one chunk.
#include "kda_device.h"
#include "kda_internal.h"

namespace kda {

namespace {

constexpr int kMaxChunks = 64;
constexpr int kManySeqs = 64;

// Per-sequence workspace record.
struct Walk {
  double spent;      // C of the last node
  int32_t node;      // the last node, -1: no nodes
  int32_t pad;
};

struct VerifyPlan {
  int chunks, chunk;        // chunks of the vocabulary, elements in each
  size_t walks, sums, total;
};

// (V <= KDA_VERIFY_MAX_VOCAB, so element indices of a row stay far inside 32 bits.)
// A chunk is one wave's work. At most 64 of them (a lane each when they are
// joined), of 4096 elements or more, or of 1024 where there are too few
// sequences to fill the GPU otherwise.
VerifyPlan verify_plan(int32_t N, int32_t V) {
  VerifyPlan p;
  const int least = N >= kManySeqs ? 4096 : 1024;
  const int chunk = ((V + kMaxChunks - 1) / kMaxChunks + 7) / 8 * 8;
  p.chunk = chunk < least ? least : chunk;
  p.chunks = (V + p.chunk - 1) / p.chunk;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  p.walks = 0;
  p.sums = up(sizeof(Walk) * (size_t)N);
  p.total = p.sums + up(2 * sizeof(double) * (size_t)N * p.chunks);
  return p;
}

// Whether one workgroup per sequence does all of it (whole_kernel), or the
// rows are spread over the GPU (walk, sums, choose). The first saves one or two
// launches and a second read of the nodes; the second is faster where few
// compute units would read long rows, or where the sequences are more than the
// 256 compute units that each hold one such workgroup. In trees with draft rows
// the walk itself takes one workgroup per sequence, so there is less to spread.
// Measured, T = 6, whole / spread in us, * where the rule takes the slower one by
// more than 2 us:
//   fp32                 N 8      48       160      256      320      1024
//   chains, draft rows
//     V  16384           15/18    15/18    15/18    15/17    21/19    46/38
//     V  49152           23/27    17/17    19/20    23/26    36/31    83/77
//     V 131072           26/17    29/17    36/37    48/51    76/62    174/172
//   chains or trees without draft rows
//     V  16384           15/18    15/18    15/17    15/18    19/19    38/29
//     V  49152           22/27    15/16    17/19    18/22    29/25    61/48
//     V 131072           22/17    25/16    28/26    34/34    53/41    116/98
//   trees, draft rows
//     V  16384           18/21    21/24    23/29    24/30    28/34    61/59
//     V  49152           26/25    35/37    35/44    42/52    46/56    107/117
//     V 131072           57/52    48/54    67/81    78/93    94/104   229/243
//   bf16
//   chains, draft rows
//     V  16384           14/17    14/17    15/17    14/17    22/17    44/24
//     V  49152           16/17    17/17    18/17    19/20    31/22    67/45
//     V 131072           21/17    22/17    25/25    29/32    48/37    107/91
//   chains or trees without draft rows
//     V  16384           14/16    14/16    14/16    14/17    22/18    42/24
//     V  49152           16/16    16/17    17/18    18/19    28/21    58/38
//     V 131072           21/17    21/17    24/22    26/27    41/31    88/66
//   trees, draft rows
//     V  16384           24/25    31/32    35/37    35/37    38/39    79/66*
//     V  49152           28/25*   38/37    35/37    39/43    45/47    97/85*
//     V 131072           60/52    48/45*   61/64    65/70    76/75    149/140*
// The borders at long rows: chains with draft rows, V 65536, fp32: N 128 22/21,
// 160 23/24; trees, V 65536: N 8 26/25, V 131072: N 32 52/52.
bool whole(int32_t N, int32_t V, bool sampled_tree) {
  if (sampled_tree) return V <= 65536 || N >= 32;
  return N <= 256 && (V <= 49152 || N >= 160);
}

// A stored probability; whatever is no finite positive number counts as 0.
template <typename T>
__device__ __forceinline__ double weight(T raw) {
  const float x = Elem<T>::load(&raw);
  constexpr int kPositive = 1 << 7 | 1 << 8;            // classes: subnormal and normal above 0
  float y = __builtin_amdgcn_classf(x, kPositive) ? x : 0.f;
  asm("" : "+v"(y));             // selected in 32 bits, not after the conversion in 64
  return (double)y;
}

__device__ __forceinline__ double lane_xor64(double x, int m) { return __shfl_xor(x, m); }
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) x += lane_xor64(x, m);
  return x;
}

// The tree of one sequence as a wave holds it: lane t is node t.
template <typename T>
struct Nodes {
  int parent, token;
  double p, q, u;     // target and draft probability of the node's token at its parent
};

template <typename T>
__device__ __forceinline__ Nodes<T> load_nodes(const T* target, const T* draft, const int32_t* tokens,
                                               const int32_t* parents, const float* uniforms, size_t n, int T_, int nt,
                                               int V, int lane) {
  Nodes<T> d;
  d.parent = -1; d.token = -1; d.p = 0.0; d.q = draft ? 0.0 : 1.0; d.u = 1.0;
  if (lane >= 1 && lane < nt) {
    const size_t at = n * T_ + lane;
    d.token = tokens[at];
    d.parent = parents ? parents[at] : lane - 1;
    d.u = (double)uniforms[at];
    if (d.parent < 0 || d.parent >= lane) d.parent = -1;
    if (d.parent >= 0 && d.token >= 0 && d.token < V) {
      const size_t e = (n * T_ + d.parent) * (size_t)V + d.token;
      d.p = weight<T>(target[e]);
      if (draft) d.q = weight<T>(draft[e]);
    } else if (d.parent >= 0 && draft == nullptr) {
      d.q = 1.0;
    }
  }
  return d;
}

// One element's residual weight, rounded the same wherever it is formed (a sum
// above 0 has an element above 0). Mode without draft: the rejected tokens are
// taken out by the callers.
__device__ __forceinline__ double residual(double p, double q, double spent) { return fmax(fma(-spent, q, p), 0.0); }

// Walks one sequence's tree; every lane of the calling wave returns the same.
// mass(cur, spent): sum of the residual row of node cur, for a node with
// another child to test (only with draft rows).
template <typename T, typename Mass>
__device__ __forceinline__ void walk(const Nodes<T>& d, bool has_draft, int nt, int lane, int& cur, int& count,
                                     double& spent, uint64_t& accepted, Mass&& mass) {
  cur = 0; count = 1; spent = 0.0;
  accepted = 1;
  double c = 1.0;
  uint64_t gone = 0;            // rejected children of cur
  uint64_t kids = __ballot(d.parent == 0);
  while (kids) {
    const int t = __builtin_ctzll(kids);
    kids &= kids - 1;
    const double p = __shfl(d.p, t), q = __shfl(d.q, t), u = __shfl(d.u, t);
    const int x = __shfl(d.token, t);
    double r;
    if (has_draft) r = residual(p, q, spent);
    else r = __ballot(d.token == x) & gone ? 0.0 : p;
    if (u * q * c < r) {
      cur = t;
      ++count;
      accepted |= 1ull << t;
      spent = 0.0; c = 1.0; gone = 0;
      kids = __ballot(d.parent == t);
    } else if (has_draft) {
      spent += c;
      if (kids) c = mass(cur, spent);
    } else {
      c -= r;
      gone |= 1ull << t;
    }
  }
}

__device__ __forceinline__ int node_count(const int32_t* num_nodes, uint32_t n, int T) {
  return num_nodes ? min(max(num_nodes[n], 0), T) : T;
}

// Results of the walk: accept, path, and the record for the later kernels.
__device__ __forceinline__ void write_walk(int lane, size_t n, int T, int nt, int cur, int count, double spent,
                                           uint64_t accepted, int32_t* accept, int32_t* path, int32_t* next_token,
                                           Walk* walks) {
  if (nt == 0) { cur = -1; count = 0; accepted = 0; }
  if (lane < T) {
    // lane's accepted node goes to the place of its rank; places past the path hold -1
    if (accepted >> lane & 1) path[n * T + __builtin_popcountll(accepted & ((1ull << lane) - 1))] = lane;
    if (lane >= count) path[n * T + lane] = -1;
  }
  if (lane == 0) {
    accept[n] = count;
    if (nt == 0) next_token[n] = -1;
    walks[n].spent = spent;
    walks[n].node = cur;
  }
}

// Rows start at any element (V may be odd). They are read in groups of 16
// bytes at aligned addresses: group i of a range [a, b) starts at element
// a - skew(a) + i * kPer, and elements outside [a, b) are never read.
template <typename T>
constexpr int kPer = 16 / sizeof(T);
template <typename T>
__device__ __forceinline__ int skew(const T* at) { return (int)(((uintptr_t)at / sizeof(T)) % kPer<T>); }

template <typename T>
__device__ __forceinline__ void load_group(const T* row, int first, int a, int b, double (&w)[kPer<T>]) {
  if (first >= a && first <= b - kPer<T>) {
    T x[kPer<T>];
    *(u32x4*)x = *(const u32x4*)(row + first);
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) w[j] = weight<T>(x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer<T>; ++j) w[j] = first + j >= a && first + j < b ? weight<T>(row[first + j]) : 0.0;
  }
}

// 16 bytes; kOnce: of a row that is read once, past the caches (the sums over
// 256 x 2 rows of 131072: 57 us through them, 50 us past them, 5.3 TB/s).
template <bool kOnce, typename T>
__device__ __forceinline__ u32x4 load16(const T* p) {
  if constexpr (kOnce) return __builtin_nontemporal_load((const u32x4*)p);
  else return *(const u32x4*)p;
}

// f(element, p, q) for the elements of [a, b) that fall to thread tid of
// `threads` (kQ = false: q is 0). Aligned groups run eight at a time with all
// their loads in flight, the rest four at a time: a group past the end is
// loaded again from the last one with its values dropped, so there is no
// branch between the loads, and f is called by all lanes together.
template <bool kQ, bool kOnce, typename T, typename F>
__device__ __forceinline__ void for_range(const T* p, const T* q, int a, int b, int tid, int threads, F&& f) {
  const int head = min((kPer<T> - skew(p + a)) % kPer<T>, b - a);
  const int groups = (b - a - head) / kPer<T>;
  const T *pg = p + a + head, *qg = kQ ? q + a + head : nullptr;
  auto some = [&](int base, auto Unroll, auto Whole) __attribute__((always_inline)) {
    constexpr int kUnroll = decltype(Unroll)::value;
    constexpr bool kWhole = decltype(Whole)::value;
    u32x4 x[kUnroll], y[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = base + tid + k * threads, at = kWhole ? i : min(i, groups - 1);
      x[k] = load16<kOnce>(pg + at * kPer<T>);
      if (kQ) y[k] = load16<kOnce>(qg + at * kPer<T>);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int i = base + tid + k * threads;
      if (!kWhole && i >= groups) x[k] = u32x4{0, 0, 0, 0};
      T u[kPer<T>], w[kPer<T>];
      *(u32x4*)u = x[k];
      if (kQ) *(u32x4*)w = y[k];
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j)
        f(a + head + i * kPer<T> + j, weight<T>(u[j]), kQ ? weight<T>(w[j]) : 0.0);
      if (!kOnce) __builtin_amdgcn_sched_barrier(0);   // one group's fp64 values at a time
    }
  };
  int base = 0;
  for (; base + 8 * threads <= groups; base += 8 * threads)
    some(base, std::integral_constant<int, 8>{}, std::true_type{});
  constexpr int kRest = kOnce ? 4 : 8;   // a walk's sum is one round trip to memory
#pragma unroll 1
  for (; base < groups; base += kRest * threads) some(base, std::integral_constant<int, kRest>{}, std::false_type{});
  const int tail = a + head + groups * kPer<T>;
  const int x = tid < head ? a + tid : tail + (tid - head);     // fewer than 2 kPer, all in one turn
  double wp = 0.0, wq = 0.0;
  if (x < b && tid < 2 * kPer<T>) {
    wp = weight<T>(p[x]);
    if (kQ) wq = weight<T>(q[x]);
  }
  f(x, wp, wq);
}

// The rejected tokens of the last node without draft rows: the tokens of its
// children (had one been accepted, it would be the last node). Lane t: node
// t's token, or -1.
__device__ __forceinline__ int gone_token(const int32_t* tokens, const int32_t* parents, size_t n, int T, int nt,
                                          int cur, int lane) {
  if (lane <= cur || lane >= nt) return -1;
  const size_t at = n * T + lane;
  return (parents ? parents[at] : lane - 1) == cur ? tokens[at] : -1;
}
struct Gone {
  int count;
  int token[kWave];
};
// Called by one wave; other waves read `gone` after a barrier.
__device__ __forceinline__ void list_gone(Gone& gone, int x, int lane) {
  const uint64_t mask = __ballot(x >= 0);
  if (x >= 0) gone.token[__builtin_popcountll(mask & ((1ull << lane) - 1))] = x;
  if (lane == 0) gone.count = __builtin_popcountll(mask);
}
__device__ __forceinline__ bool is_gone(const Gone& gone, int x) {
  for (int i = 0; i < gone.count; ++i)
    if (gone.token[i] == x) return true;
  return false;
}

// The walk of a tree with draft rows: a workgroup per sequence, since masses
// are sums over rows. Every wave walks; the sums are shared through LDS in a
// fixed order, so all waves take the same turns.
constexpr int kWalkThreads = 1024;
template <typename T>
struct Mass {
  const T *target, *draft;
  uint32_t n;
  int T_, V, tid, turn = 0;
  __device__ __forceinline__ double operator()(int at, double C) {
    __shared__ double s_sum[2][kWalkThreads / kWave];
    const size_t row = ((size_t)n * T_ + at) * (size_t)V;
    double sum = 0.0;
    for_range<true, false>(target + row, draft + row, 0, V, tid, kWalkThreads,
                           [&](int, double p, double q) { sum += residual(p, q, C); });
    sum = wave_sum(sum);
    // two buffers in turn: a wave may start the next sum while another still
    // reads this one, but not the one after it
    if (tid % kWave == 0) s_sum[turn][tid / kWave] = sum;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < kWalkThreads / kWave; ++w) total += s_sum[turn][w];
    turn ^= 1;
    return total;
  }
};

template <typename T>
__global__ __launch_bounds__(kWalkThreads) void walk_kernel(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes,
    const float* __restrict__ uniforms, int32_t* __restrict__ accept, int32_t* __restrict__ path,
    int32_t* __restrict__ next_token, int T_, int V, Walk* __restrict__ walks) {
  const uint32_t n = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int nt = node_count(num_nodes, n, T_);
  const Nodes<T> d = load_nodes<T>(target, draft, tokens, parents, uniforms, n, T_, nt, V, lane);
  int cur, count;
  double spent;
  uint64_t accepted;
  Mass<T> mass{target, draft, n, T_, V, tid};
  walk<T>(d, true, nt, lane, cur, count, spent, accepted, [&](int at, double C) { return mass(at, C); });
  if (wave == 0) write_walk(lane, n, T_, nt, cur, count, spent, accepted, accept, path, next_token, walks);
}

// Sums of r and p over elements [a, b) of the last node's row, by one wave.
// gone: lane t's rejected token (without draft rows), or -1.
template <typename T, bool kDraft>
__device__ __forceinline__ void wave_sums(const T* p, const T* q, double spent, int gone, int a, int b, int lane,
                                          double& rs, double& ps) {
  rs = ps = 0.0;
  const uint64_t here = kDraft ? 0 : __ballot(gone >= a && gone < b);
  if (kDraft && spent > 0.0)            // (the row of q matters only after a rejection)
    for_range<true, true>(p, q, a, b, lane, kWave, [&](int, double x, double y) {
      rs += residual(x, y, spent);
      ps += x;
    });
  else if (here)
    for_range<false, true>(p, (const T*)nullptr, a, b, lane, kWave, [&](int at, double x, double) {
      bool out = false;
      for (uint64_t m = here; m; m &= m - 1) out |= at == __builtin_amdgcn_readlane(gone, __builtin_ctzll(m));
      rs += out ? 0.0 : x;
      ps += x;
    });
  else
    for_range<false, true>(p, (const T*)nullptr, a, b, lane, kWave, [&](int, double x, double) { ps += x; });
  if (!(kDraft && spent > 0.0) && !here) rs = ps;
  rs = wave_sum(rs);
  ps = wave_sum(ps);
}

// Partial sums of the last node's r (and of p, for the case that r is 0
// everywhere), one chunk per wave. kWalk: no masses are needed (chains, or no
// draft rows), so every wave walks by itself, and the sequence's first one
// writes the results.
template <typename T, bool kDraft, bool kWalk>
__global__ __launch_bounds__(256) void sums_kernel(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes,
    const float* __restrict__ uniforms, int32_t* __restrict__ accept, int32_t* __restrict__ path,
    int32_t* __restrict__ next_token, int T_, int V, int chunk, int chunks, Walk* __restrict__ walks,
    double* __restrict__ sums) {
  const uint32_t groups = (uint32_t)(chunks + 3) / 4, n = blockIdx.x / groups;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int part = (int)(blockIdx.x % groups) * 4 + wave;
  if (part >= chunks) return;
  const int nt = node_count(num_nodes, n, T_);
  int cur;
  double spent;
  if constexpr (kWalk) {
    const Nodes<T> d = load_nodes<T>(target, draft, tokens, parents, uniforms, n, T_, nt, V, lane);
    int count;
    uint64_t accepted;
    walk<T>(d, kDraft, nt, lane, cur, count, spent, accepted, [](int, double) { return 0.0; });
    if (part == 0) write_walk(lane, n, T_, nt, cur, count, spent, accepted, accept, path, next_token, walks);
  } else {
    cur = walks[n].node;
    spent = walks[n].spent;
  }
  if (nt == 0) return;
  const size_t row = ((size_t)n * T_ + cur) * (size_t)V;
  const int a = part * chunk, b = min(V - a, chunk) + a;
  const int gone = kDraft ? -1 : gone_token(tokens, parents, n, T_, nt, cur, lane);
  double rs, ps;
  wave_sums<T, kDraft>(target + row, draft + row, spent, gone, a, b, lane, rs, ps);
  if (lane < 2) sums[((size_t)n * chunks + part) * 2 + lane] = lane ? ps : rs;
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ double wave_scan(double x, int lane) {
#pragma unroll
  for (int m = 1; m < kWave; m *= 2) {
    const double y = __shfl_up(x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// The next token: the chunk where the running sum of r passes u * sum(r), then
// the token inside it. r, p: the sums of chunk `lane`. A tile of the chunk is
// kRun consecutive elements per thread. Where rounding leaves the threshold
// past the last sum, the last token with r > 0 is taken. Returns the token, in
// every thread; -1 if p is 0 everywhere.
template <typename T, bool kDraft, int kThreads, int kRun>
__device__ __forceinline__ int choose(const T* tp, const T* tq, double spent, double u, double r, double p, int gone,
                                      int V, int chunk, int tid) {
  constexpr int kWaves = kThreads / kWave;
  const int lane = tid % kWave, wave = tid / kWave;
  __shared__ double s_sum[kWaves];
  __shared__ int s_last[kWaves];
  __shared__ int s_token;
  __shared__ Gone s_gone;
  const bool plain = !(wave_sum(r) > 0.0);     // r is 0 everywhere: draw from p
  if (plain) { r = p; spent = 0.0; }
  const double upto = wave_scan(r, lane);
  const uint64_t some = __ballot(r > 0.0);
  if (!some) return -1;
  const double goal = fmax(u, 0.0) * __shfl(upto, kWave - 1);
  const uint64_t past = __ballot(upto > goal) & some;
  const int part = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
  double left = goal - __shfl(upto - r, part);

  if (!kDraft && wave == 0) list_gone(s_gone, plain ? -1 : gone, lane);
  if (tid == 0) s_token = -1;
  __syncthreads();
  if (!(kDraft && spent > 0.0)) tq = nullptr;
  const int a = part * chunk, b = min(V - a, chunk) + a;
  int last = -1;                                // last token with r > 0 so far
  for (int tile = a - skew(tp + a); tile < b; tile += kThreads * kRun) {
    const int first = tile + tid * kRun;
    double w[kRun], sum = 0.0;
    int mine = -1;
#pragma unroll
    for (int gr = 0; gr < kRun / kPer<T>; ++gr) {
      double x[kPer<T>] = {}, y[kPer<T>] = {};
      const int at = first + gr * kPer<T>;
      if (at < b) {
        load_group<T>(tp, at, a, b, x);
        if (tq) load_group<T>(tq, at, a, b, y);
      }
#pragma unroll
      for (int j = 0; j < kPer<T>; ++j) {
        double& z = w[gr * kPer<T> + j];
        z = kDraft ? residual(x[j], y[j], spent) : x[j] > 0.0 && is_gone(s_gone, at + j) ? 0.0 : x[j];
        if (z > 0.0) mine = at + j;
        sum += z;
      }
    }
    const double incl = wave_scan(sum, lane);
    int top = mine;                             // last token with r > 0 in the wave
#pragma unroll
    for (int m = 1; m < kWave; m *= 2) top = max(top, __shfl_xor(top, m));
    if (lane == kWave - 1) s_sum[wave] = incl;
    if (lane == 0) s_last[wave] = top;
    __syncthreads();
    double before = 0.0;
    for (int x = 0; x < wave; ++x) before += s_sum[x];
    double total = before;
    for (int x = wave; x < kWaves; ++x) total += s_sum[x];
    for (int x = 0; x < kWaves; ++x) last = max(last, s_last[x]);
    // the first thread whose running sum passes the threshold finds the token
    double run = before + (incl - sum);
    const bool here = before + incl > left;
    const uint64_t ok = __ballot(here && sum > 0.0);
    if (ok && lane == __builtin_ctzll(ok)) {
      int token = mine;
#pragma unroll
      for (int j = kRun - 1; j >= 0; --j) {
        // from the end: the lowest element at which the sum has passed
        double upto_j = run;
#pragma unroll
        for (int x = 0; x <= j; ++x) upto_j += w[x];
        if (upto_j > left && w[j] > 0.0) token = first + j;
      }
      atomicMin((unsigned*)&s_token, (unsigned)token);   // waves in order of tokens
    }
    __syncthreads();
    if (s_token != -1) break;
    left -= total;
    __syncthreads();
  }
  return s_token != -1 ? s_token : last;
}

template <typename T, bool kDraft>
__global__ __launch_bounds__(256) void choose_kernel(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes,
    const float* __restrict__ uniforms, int32_t* __restrict__ next_token, int T_, int V, int chunk, int chunks,
    const Walk* __restrict__ walks, const double* __restrict__ sums) {
  const uint32_t n = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int nt = node_count(num_nodes, n, T_);
  if (nt == 0) return;
  const int cur = walks[n].node;
  double r = 0.0, p = 0.0;
  if (lane < chunks) {
    r = sums[((size_t)n * chunks + lane) * 2];
    p = sums[((size_t)n * chunks + lane) * 2 + 1];
  }
  const size_t row = ((size_t)n * T_ + cur) * (size_t)V;
  const int gone = kDraft ? -1 : gone_token(tokens, parents, n, T_, nt, cur, lane);
  const int token = choose<T, kDraft, 256, 16>(target + row, draft + row, walks[n].spent,
                                               (double)uniforms[(size_t)n * T_], r, p, gone, V, chunk, tid);
  if (tid == 0) next_token[n] = token;
}

// All three steps by one workgroup per sequence: one launch, but a row passes
// through one compute unit.
template <typename T, bool kDraft>
__global__ __launch_bounds__(kWalkThreads) void whole_kernel(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ parents, const int32_t* __restrict__ num_nodes,
    const float* __restrict__ uniforms, int32_t* __restrict__ accept, int32_t* __restrict__ path,
    int32_t* __restrict__ next_token, int T_, int V, int chunk, Walk* __restrict__ walks) {
  constexpr int kWaves = kWalkThreads / kWave;
  const uint32_t n = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int nt = node_count(num_nodes, n, T_);
  __shared__ double s_part[2][kWaves];
  const Nodes<T> d = load_nodes<T>(target, draft, tokens, parents, uniforms, n, T_, nt, V, lane);
  int cur, count;
  double spent;
  uint64_t accepted;
  Mass<T> mass{target, draft, n, T_, V, tid};
  walk<T>(d, kDraft, nt, lane, cur, count, spent, accepted, [&](int at, double C) { return mass(at, C); });
  if (wave == 0) write_walk(lane, n, T_, nt, cur, count, spent, accepted, accept, path, next_token, walks);
  if (nt == 0) return;
  const size_t row = ((size_t)n * T_ + cur) * (size_t)V;
  const int gone = kDraft ? -1 : gone_token(tokens, parents, n, T_, nt, cur, lane);
  const int a = min(wave * chunk, V), b = min(V - a, chunk) + a;
  double rs, ps;
  wave_sums<T, kDraft>(target + row, draft + row, spent, gone, a, b, lane, rs, ps);
  if (lane == 0) { s_part[0][wave] = rs; s_part[1][wave] = ps; }
  __syncthreads();
  double r = 0.0, p = 0.0;
  if (lane < kWaves) { r = s_part[0][lane]; p = s_part[1][lane]; }
  const int token = choose<T, kDraft, kWalkThreads, 8>(target + row, draft + row, spent,
                                                       (double)uniforms[(size_t)n * T_], r, p, gone, V, chunk, tid);
  if (tid == 0) next_token[n] = token;
}


template <typename T>
hipError_t launch_verify_t(const VerifyArgs& a) {
  const VerifyPlan p = verify_plan(a.N, a.V);
  Walk* walks = (Walk*)((char*)a.workspace + p.walks);
  double* sums = (double*)((char*)a.workspace + p.sums);
  const T *target = (const T*)a.target, *draft = (const T*)a.draft;
  const dim3 grid((unsigned)((int64_t)a.N * ((p.chunks + 3) / 4)));
#define KDA_SUMS(DRAFT, WALK)                                                                                       \
  hipLaunchKernelGGL((sums_kernel<T, DRAFT, WALK>), grid, dim3(256), 0, a.stream, target, draft, a.tokens, a.parents, \
                     a.num_nodes, a.uniforms, a.accept, a.path, a.next_token, a.T, a.V, p.chunk, p.chunks, walks,   \
                     sums)
#define KDA_CHOOSE(DRAFT)                                                                                           \
  hipLaunchKernelGGL((choose_kernel<T, DRAFT>), dim3((unsigned)a.N), dim3(256), 0, a.stream, target, draft,         \
                     a.tokens, a.parents, a.num_nodes, a.uniforms, a.next_token, a.T, a.V, p.chunk, p.chunks,       \
                     walks, sums)
  if (whole(a.N, a.V, draft && a.parents)) {
    const int chunk = ((a.V + 15) / 16 + 7) / 8 * 8;
    if (draft)
      hipLaunchKernelGGL((whole_kernel<T, true>), dim3((unsigned)a.N), dim3(kWalkThreads), 0, a.stream, target, draft,
                         a.tokens, a.parents, a.num_nodes, a.uniforms, a.accept, a.path, a.next_token, a.T, a.V,
                         chunk, walks);
    else
      hipLaunchKernelGGL((whole_kernel<T, false>), dim3((unsigned)a.N), dim3(kWalkThreads), 0, a.stream, target,
                         draft, a.tokens, a.parents, a.num_nodes, a.uniforms, a.accept, a.path, a.next_token, a.T,
                         a.V, chunk, walks);
  } else if (draft && a.parents) {
    hipLaunchKernelGGL((walk_kernel<T>), dim3((unsigned)a.N), dim3(kWalkThreads), 0, a.stream, target, draft,
                       a.tokens, a.parents, a.num_nodes, a.uniforms, a.accept, a.path, a.next_token, a.T, a.V, walks);
    KDA_SUMS(true, false);
    KDA_CHOOSE(true);
  } else if (draft) {
    KDA_SUMS(true, true);
    KDA_CHOOSE(true);
  } else {
    KDA_SUMS(false, true);
    KDA_CHOOSE(false);
  }
#undef KDA_SUMS
#undef KDA_CHOOSE
  return hipGetLastError();
}

}  // namespace

// Grows with N and V, so that a workspace serves every smaller call too: a plan
// for fewer than 64 sequences has up to four times the chunks for each, so it may
// need more than one for a few more sequences.
size_t verify_workspace(int32_t N, int32_t T, int32_t V) {
  const size_t few = verify_plan(N < kManySeqs ? N : kManySeqs - 1, V).total, all = verify_plan(N, V).total;
  return few > all ? few : all;
}

hipError_t launch_verify(const VerifyArgs& a) {
  return a.bf16 ? launch_verify_t<bf16_bits>(a) : launch_verify_t<float>(a);
}

}  // namespace kda
