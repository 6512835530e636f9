// C ABI of libkda (declared in include/kda.h): argument validation, workspace
// sizing and dispatch to the kernel launchers. No device work is enqueued
// unless every argument checks out.
#include "kda.h"
#include "kda_internal.h"
#include "kda_plan.h"

#include <float.h>
#include <limits.h>
#include <string.h>

#include <initializer_list>

namespace {

bool supported_dims(int32_t Dk, int32_t Dv) { return Dk == Dv && (Dk == 16 || Dk == 128); }

// An enum argument as the int a C caller passed. A C enum is an int, but in
// C++ a value outside the enumerators' range may not be read as the enum type,
// so the argument's bytes are read instead (by reference: no enum-typed load).
template <typename E>
int enum_code(const E& e) {
  static_assert(sizeof(E) == sizeof(int), "C enums are int-sized");
  int c;
  memcpy(&c, &e, sizeof c);
  return c;
}

// Validates cu_seqlens_host; on success returns total tokens and prefill
// blocks (kda::kBlockTokens tokens each).
bool scan_lengths(const int32_t* cu, int32_t num_seqs, int64_t* tokens, int64_t* blocks) {
  if (!cu || num_seqs < 0 || cu[0] != 0) return false;
  int64_t c = 0;
  for (int32_t n = 0; n < num_seqs; ++n) {
    if (cu[n + 1] < cu[n]) return false;
    c += (cu[n + 1] - cu[n] + kda::kBlockTokens - 1) / kda::kBlockTokens;
  }
  *tokens = cu[num_seqs];
  *blocks = c;
  return c <= INT32_MAX;
}

kda_status from_hip(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// Lowest decay floor the prefill accepts: a chunk's decayed keys span a
// factor of up to exp(-16 g_min) (k / P_r with P_r >= exp(16 g_min) inside
// each 16-token chunk), which must stay inside the fp32 / bf16 normal range
// (2^126) with margin.
constexpr float kMinGateFloor = KDA_PREFILL_MIN_G_FLOOR;
static_assert(KDA_CHUNK * -KDA_PREFILL_MIN_G_FLOOR * 1.4426950408889634f < 120.f,
              "decay span of a chunk");

// Options: NULL, or known flag bits, a known gate layout and a usable epsilon.
bool options_ok(const kda_options* opt) {
  if (!opt) return true;
  const uint32_t known = KDA_FE_L2NORM_QK | KDA_FE_GATE_LOGITS | KDA_FE_BETA_LOGITS;
  if (opt->flags & ~known) return false;
  if (opt->gate != KDA_GATE_CHANNEL && opt->gate != KDA_GATE_HEAD && opt->gate != KDA_GATE_NONE) return false;
  if (opt->gate == KDA_GATE_NONE && (opt->flags & KDA_FE_GATE_LOGITS)) return false;
  if (opt->segments < 0 || opt->segments > KDA_MAX_SEGMENTS) return false;
  return opt->norm_eps >= 0.f && opt->norm_eps <= FLT_MAX;
}
int32_t gate_of(const kda_options* opt) { return opt ? opt->gate : KDA_GATE_CHANNEL; }

// Decode multiplies the state by alpha = exp(clamp(g, g_min, 0)) directly, so
// any finite floor at or below 0 is usable.
bool decode_floor_ok(float g_min) { return g_min >= -FLT_MAX && g_min <= 0.f; }

kda_status prefill_impl(const void* q, const void* k, const void* v, int dtype, const float* g,
                        const float* beta, const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                        int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv, float scale, float g_min,
                        const float* initial_state, float* final_state, int32_t ckpt_interval,
                        float* checkpoints, void* o, void* workspace, size_t workspace_bytes,
                        bool use_scratch, const kda_options* opt, hipStream_t stream);

// Every tensor pointer must be 16-byte aligned (NULL passes).
bool aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15) return false;
  return true;
}

// Arrays read one 4-byte element at a time need their natural alignment only.
bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 3) return false;
  return true;
}

// An array as a call uses it (p NULL: not used).
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  return a.p && b.p && (uintptr_t)a.p < (uintptr_t)b.p + b.bytes && (uintptr_t)b.p < (uintptr_t)a.p + a.bytes;
}
// Whether no array that is written shares a byte with another one of the call.
bool apart(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* x = w + 1; x != written.end(); ++x)
      if (overlap(*w, *x)) return false;
    for (const Span& r : read)
      if (overlap(*w, r)) return false;
  }
  return true;
}

}  // namespace

extern "C" {

const char* kda_status_string(kda_status status) {
  switch (enum_code(status)) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG: invalid argument";
    case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED: unsupported head size or dtype";
    case KDA_ERR_WORKSPACE: return "KDA_ERR_WORKSPACE: workspace missing or too small";
    case KDA_ERR_HIP: return "KDA_ERR_HIP: HIP runtime error";
  }
  return "KDA: unknown status";
}

int64_t kda_prefill_num_checkpoints(const int32_t* cu_seqlens_host, int32_t num_seqs,
                                    int32_t ckpt_interval) {
  int64_t tokens, blocks;
  if (!scan_lengths(cu_seqlens_host, num_seqs, &tokens, &blocks)) return -1;
  if (ckpt_interval <= 0) return 0;
  int64_t total = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    total += (cu_seqlens_host[n + 1] - cu_seqlens_host[n]) / ckpt_interval;
  return total;
}

size_t kda_prefill_workspace_size_window(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t Dk,
                                         int32_t Dv, int64_t window_blocks) {
  if (num_seqs < 0 || total_tokens < 0 || H <= 0 || !supported_dims(Dk, Dv) || window_blocks <= 0) return 0;
  // shapes the prefill refuses (token-heads or 16-column slices past INT32_MAX)
  if (total_tokens > INT32_MAX || total_tokens * H > INT32_MAX || (int64_t)num_seqs * H * (Dv / 16) > INT32_MAX)
    return 0;
  // sum_n ceil(L_n / 32) <= sum_n (L_n / 32 + 1) for any lengths with this total
  const int64_t max_blocks = total_tokens / kda::kBlockTokens + num_seqs;
  if (max_blocks > INT32_MAX) return 0;
  const bool windowed = window_blocks < max_blocks;
  return kda::prefill_layout(num_seqs, max_blocks, H, Dk, windowed ? window_blocks : max_blocks, windowed).total;
}

size_t kda_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t Dk,
                                  int32_t Dv) {
  if (H <= 0 || !supported_dims(Dk, Dv)) return 0;
  const size_t cap_bytes = num_seqs == 1 ? (size_t)KDA_PREFILL_SINGLE_SEQ_WINDOW_BYTES
                                         : (size_t)KDA_PREFILL_RECORD_CAP_BYTES;
  const int64_t cap = (int64_t)(cap_bytes / (kda::record_bytes(Dk) * (size_t)H));
  return kda_prefill_workspace_size_window(num_seqs, total_tokens, H, Dk, Dv, cap > 1 ? cap : 1);
}

kda_status kda_prefill_chunked(const void* q, const void* k, const void* v, kda_dtype dtype,
                               const float* g, const float* beta, const int32_t* cu_seqlens,
                               const int32_t* cu_seqlens_host, int32_t num_seqs, int32_t H,
                               int32_t Dk, int32_t Dv, float scale, float g_min,
                               const float* initial_state, float* final_state,
                               int32_t ckpt_interval, float* checkpoints, void* o,
                               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return prefill_impl(q, k, v, enum_code(dtype), g, beta, cu_seqlens, cu_seqlens_host, num_seqs, H, Dk, Dv,
                      scale, g_min, initial_state, final_state, ckpt_interval, checkpoints, o, workspace,
                      workspace_bytes, false, nullptr, stream);
}

}  // extern "C"

namespace {

// The prefill behind both workspace conventions: the caller's workspace, or
// (use_scratch) the library's static per-device scratch, looked up only after
// every argument and the size have been checked.
kda_status prefill_impl(const void* q, const void* k, const void* v, int dtype, const float* g,
                        const float* beta, const int32_t* cu_seqlens, const int32_t* cu_seqlens_host,
                        int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv, float scale, float g_min,
                        const float* initial_state, float* final_state, int32_t ckpt_interval,
                        float* checkpoints, void* o, void* workspace, size_t workspace_bytes,
                        bool use_scratch, const kda_options* opt, hipStream_t stream) {
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!options_ok(opt)) return KDA_ERR_INVALID_ARG;
  const bool need_g = gate_of(opt) != KDA_GATE_NONE;
  if (!supported_dims(Dk, Dv)) return KDA_ERR_UNSUPPORTED;
  int64_t tokens, blocks;
  if (H <= 0 || num_seqs < 0 || !cu_seqlens || !scan_lengths(cu_seqlens_host, num_seqs, &tokens, &blocks))
    return KDA_ERR_INVALID_ARG;
  if (!(g_min >= kMinGateFloor && g_min <= 0.f)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)num_seqs * H * (Dv / 16) > INT32_MAX || tokens * (int64_t)H > INT32_MAX)
    return KDA_ERR_INVALID_ARG;
  if (tokens > 0 && (!q || !k || !v || (need_g && !g) || !beta || !o)) return KDA_ERR_INVALID_ARG;
  if (ckpt_interval < 0 || (ckpt_interval > 0 && ckpt_interval % KDA_CHUNK != 0))
    return KDA_ERR_INVALID_ARG;
  const int64_t nck = kda_prefill_num_checkpoints(cu_seqlens_host, num_seqs, ckpt_interval);
  if (nck > 0 && !checkpoints) return KDA_ERR_INVALID_ARG;
  if (!aligned16({q, k, v, g, beta, cu_seqlens, initial_state, final_state, checkpoints, o}))
    return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  // segments per sequence: the library's choice (0), off (1), or forced
  // (where the workspace holds the segment states)
  const int32_t req = opt ? opt->segments : 0;
  if (req >= 2 && !kda::segments_allowed(num_seqs, H, Dk)) return KDA_ERR_INVALID_ARG;
  // Record windows: all of the call's records at once if the workspace holds
  // them, else windows of as many blocks as it holds, evened out.
  // A window also keeps the prep grid's second dimension (its blocks) within
  // kMaxWindowBlocks.
  constexpr int64_t kMaxWindowBlocks = 65535;
  // A single sequence runs in windows of about
  // KDA_PREFILL_SINGLE_SEQ_WINDOW_BYTES of records even when the workspace
  // holds more: every window then still holds all of its (sequence, head)
  // pairs, and part of each window's records is still in the memory-side
  // cache when the chain reads them.
  const size_t rec_bytes = kda::record_bytes(Dk) * (size_t)H;
  int64_t max_window = kMaxWindowBlocks;
  if (num_seqs == 1) {
    const int64_t w1 = (int64_t)((size_t)KDA_PREFILL_SINGLE_SEQ_WINDOW_BYTES / rec_bytes);
    max_window = w1 < 1 ? 1 : (w1 < max_window ? w1 : max_window);
  }
  if (use_scratch) workspace_bytes = KDA_NOALLOC_SCRATCH_BYTES;
  // (every sequence empty: no records, the tables only)
  int64_t window = 1;
  if (blocks == 0) {
    if (workspace_bytes < kda::prefill_layout(num_seqs, 0, H, Dk, 0, false).total) return KDA_ERR_WORKSPACE;
  } else {
    window = kda::plan::choose_window(blocks, workspace_bytes,
                                      kda::prefill_layout(num_seqs, blocks, H, Dk, blocks, false).total,
                                      kda::prefill_layout(num_seqs, blocks, H, Dk, 0, true).total, rec_bytes,
                                      max_window);
    if (window < 1) return KDA_ERR_WORKSPACE;
  }
  if (use_scratch) {
    // the scratch of the device the work runs on: the stream's, which must be
    // the current one (the array's address is looked up with it current)
    int cur = -1, dev = -1;
    if (hipGetDevice(&cur) != hipSuccess || hipStreamGetDevice(stream, &dev) != hipSuccess) return KDA_ERR_HIP;
    if (dev != cur) return KDA_ERR_INVALID_ARG;
    if (kda::noalloc_scratch(&workspace) != hipSuccess) return KDA_ERR_HIP;
  }
  if (!workspace || ((uintptr_t)workspace & 255)) return KDA_ERR_WORKSPACE;

  kda::PrefillArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.cu_seqlens = cu_seqlens; a.cu_seqlens_host = cu_seqlens_host;
  a.num_seqs = num_seqs; a.H = H; a.D = Dk;
  a.total_tokens = tokens; a.total_blocks = blocks; a.window_blocks = window;
  a.num_checkpoints = nck > 0 ? nck : 0;
  a.scale = scale; a.g_min = g_min;
  a.fe_flags = opt ? opt->flags : 0u; a.fe_eps = opt ? opt->norm_eps : 0.f;
  a.gate = gate_of(opt);
  a.segments = req;
  a.initial_state = initial_state; a.final_state = final_state;
  a.ckpt_interval = nck > 0 ? ckpt_interval : 0;
  a.checkpoints = checkpoints;
  a.o = o; a.workspace = workspace;
  a.bf16 = dtype == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_prefill(a));
}

}  // namespace

extern "C" {

kda_status kda_prefill_chunked_ex(const void* q, const void* k, const void* v, kda_dtype dtype,
                                  const float* g, const float* beta, const int32_t* cu_seqlens,
                                  const int32_t* cu_seqlens_host, int32_t num_seqs, int32_t H,
                                  int32_t Dk, int32_t Dv, float scale, float g_min,
                                  const float* initial_state, float* final_state,
                                  int32_t ckpt_interval, float* checkpoints, void* o,
                                  void* workspace, size_t workspace_bytes,
                                  const kda_options* opt, hipStream_t stream) {
  return prefill_impl(q, k, v, enum_code(dtype), g, beta, cu_seqlens, cu_seqlens_host, num_seqs, H, Dk, Dv, scale,
                      g_min, initial_state, final_state, ckpt_interval, checkpoints, o, workspace,
                      workspace_bytes, false, opt, stream);
}

kda_status kda_prefill_chunked_noalloc(const void* q, const void* k, const void* v, kda_dtype dtype,
                                       const float* g, const float* beta, const int32_t* cu_seqlens,
                                       const int32_t* cu_seqlens_host, int32_t num_seqs, int32_t H,
                                       int32_t Dk, int32_t Dv, float scale, float g_min,
                                       const float* initial_state, float* final_state,
                                       int32_t ckpt_interval, float* checkpoints, void* o,
                                       const kda_options* opt, hipStream_t stream) {
  return prefill_impl(q, k, v, enum_code(dtype), g, beta, cu_seqlens, cu_seqlens_host, num_seqs, H, Dk, Dv, scale,
                      g_min, initial_state, final_state, ckpt_interval, checkpoints, o, nullptr, 0, true,
                      opt, stream);
}

kda_status kda_decode_step(const void* q, const void* k, const void* v, kda_dtype dtype,
                           const float* g, const float* beta, float* state, void* o, int32_t N,
                           int32_t H, int32_t Dk, int32_t Dv, float scale, float g_min,
                           hipStream_t stream) {
  const int dt = enum_code(dtype);
  if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!supported_dims(Dk, Dv)) return KDA_ERR_UNSUPPORTED;
  if (N < 0 || H <= 0 || (int64_t)N * H > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (!decode_floor_ok(g_min)) return KDA_ERR_INVALID_ARG;
  if (N == 0) return KDA_OK;
  if (!q || !k || !v || !g || !beta || !state || !o) return KDA_ERR_INVALID_ARG;
  if (!aligned16({q, k, v, g, beta, state, o})) return KDA_ERR_INVALID_ARG;
  kda::DecodeArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.o = o;
  a.N = N; a.H = H; a.D = Dk;
  a.T = 1; a.accept = nullptr;
  a.scale = scale; a.g_min = g_min;
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_decode(a));
}

kda_status kda_decode_tokens(const void* q, const void* k, const void* v, kda_dtype dtype,
                             const float* g, const float* beta, float* state,
                             const int32_t* accept, void* o, int32_t N, int32_t T, int32_t H,
                             int32_t Dk, int32_t Dv, float scale, float g_min,
                             const kda_options* opt, hipStream_t stream) {
  const int dt = enum_code(dtype);
  if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!options_ok(opt)) return KDA_ERR_INVALID_ARG;
  const bool need_g = gate_of(opt) != KDA_GATE_NONE;
  if (!supported_dims(Dk, Dv)) return KDA_ERR_UNSUPPORTED;
  if (T < 1 || T > KDA_DECODE_MAX_TOKENS) return KDA_ERR_INVALID_ARG;
  if (!decode_floor_ok(g_min)) return KDA_ERR_INVALID_ARG;
  if (N < 0 || H <= 0 || (int64_t)N * H > INT32_MAX || (int64_t)N * T * H > INT32_MAX)
    return KDA_ERR_INVALID_ARG;
  if (N == 0) return KDA_OK;
  if (!q || !k || !v || (need_g && !g) || !beta || !state || !o) return KDA_ERR_INVALID_ARG;
  if (!aligned16({q, k, v, g, beta, state, o})) return KDA_ERR_INVALID_ARG;
  kda::DecodeArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.o = o;
  a.N = N; a.H = H; a.D = Dk;
  a.T = T; a.accept = accept;
  a.scale = scale; a.g_min = g_min;
  a.fe_flags = opt ? opt->flags : 0u; a.fe_eps = opt ? opt->norm_eps : 0.f;
  a.gate = gate_of(opt);
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_decode(a));
}

// A launch takes fewer than 2^32 threads: one workgroup of 256 per head (of 512
// for larger trees of larger heads), or of 1024 per sequence (and up to 16 of
// 256) of a verification.
constexpr int64_t kMaxHeads = KDA_MAX_LAUNCH_HEADS, kMaxTreeHeads = KDA_MAX_LARGE_TREE_HEADS;
static_assert(kMaxHeads * kda::kHeadThreads < 1ll << 32, "workgroups of the tree, commit and cache kernels");
static_assert(kMaxTreeHeads * kda::kLargeTreeThreads < 1ll << 32, "workgroups of the tree kernels of 512 threads");
static_assert(KDA_VERIFY_MAX_SEQS * 1024ll < 1ll << 32 && KDA_VERIFY_MAX_SEQS * 16ll * 256 < 1ll << 32,
              "workgroups of the verification kernels");

// Tree step: the checks kda_decode_tree and kda_commit_path share, in the order
// of kda_decode_tokens.
namespace {
kda_status tree_args_ok(int dt, const kda_options* opt, int32_t N, int32_t T, int32_t H, int32_t Dk,
                        int32_t Dv, float g_min) {
  if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!options_ok(opt)) return KDA_ERR_INVALID_ARG;
  if (!supported_dims(Dk, Dv)) return KDA_ERR_UNSUPPORTED;
  if (T < 1 || T > KDA_TREE_MAX_NODES) return KDA_ERR_INVALID_ARG;
  if (!decode_floor_ok(g_min)) return KDA_ERR_INVALID_ARG;
  if (N < 0 || H <= 0 || (int64_t)N * H > kMaxHeads || (int64_t)N * T * H > INT32_MAX)
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

bool verify_sizes_ok(int32_t N, int32_t T, int32_t V) {
  return N >= 0 && N <= KDA_VERIFY_MAX_SEQS && T >= 1 && T <= KDA_TREE_MAX_NODES && V >= 1 &&
         V <= KDA_VERIFY_MAX_VOCAB;
}
}  // namespace

kda_status kda_decode_tree(const void* q, const void* k, const void* v, kda_dtype dtype,
                           const float* g, const float* beta, const float* state,
                           const int32_t* parents, const int32_t* num_nodes, void* o, int32_t N,
                           int32_t T, int32_t H, int32_t Dk, int32_t Dv, float scale, float g_min,
                           const kda_options* opt, hipStream_t stream) {
  const int dt = enum_code(dtype);
  const kda_status st = tree_args_ok(dt, opt, N, T, H, Dk, Dv, g_min);
  if (st != KDA_OK || N == 0) return st;
  if (Dk == 128 && T > 16 && (int64_t)N * H > kMaxTreeHeads) return KDA_ERR_INVALID_ARG;
  const bool need_g = gate_of(opt) != KDA_GATE_NONE;
  if (!q || !k || !v || (need_g && !g) || !beta || !state || !o) return KDA_ERR_INVALID_ARG;
  if (!aligned16({q, k, v, g, beta, state, o}) || !aligned4({parents, num_nodes})) return KDA_ERR_INVALID_ARG;
  kda::TreeArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = const_cast<float*>(state); a.o = o;
  a.parents = parents; a.num_nodes = num_nodes;
  a.path = nullptr; a.accept = nullptr;
  a.N = N; a.T = T; a.H = H; a.D = Dk;
  a.scale = scale; a.g_min = g_min;
  a.fe_flags = opt ? opt->flags : 0u; a.fe_eps = opt ? opt->norm_eps : 0.f;
  a.gate = gate_of(opt);
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_tree(a));
}

kda_status kda_commit_path(const void* k, const void* v, kda_dtype dtype, const float* g,
                           const float* beta, float* state, const int32_t* path,
                           const int32_t* accept, int32_t N, int32_t T, int32_t H, int32_t Dk,
                           int32_t Dv, float g_min, const kda_options* opt, hipStream_t stream) {
  const int dt = enum_code(dtype);
  const kda_status st = tree_args_ok(dt, opt, N, T, H, Dk, Dv, g_min);
  if (st != KDA_OK || N == 0) return st;
  const bool need_g = gate_of(opt) != KDA_GATE_NONE;
  if (!k || !v || (need_g && !g) || !beta || !state || !path || !accept) return KDA_ERR_INVALID_ARG;
  if (!aligned16({k, v, g, beta, state}) || !aligned4({path, accept})) return KDA_ERR_INVALID_ARG;
  kda::TreeArgs a;
  a.q = nullptr; a.k = k; a.v = v; a.g = g; a.beta = beta; a.state = state; a.o = nullptr;
  a.parents = nullptr; a.num_nodes = nullptr;
  a.path = path; a.accept = accept;
  a.N = N; a.T = T; a.H = H; a.D = Dk;
  a.scale = 1.f; a.g_min = g_min;
  a.fe_flags = opt ? opt->flags : 0u; a.fe_eps = opt ? opt->norm_eps : 0.f;
  a.gate = gate_of(opt);
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_commit(a));
}

size_t kda_verify_workspace_size(int32_t N, int32_t T, int32_t V) {
  if (!verify_sizes_ok(N, T, V)) return 0;
  return kda::verify_workspace(N, T, V);
}

kda_status kda_verify_drafts(const void* target, const void* draft, kda_dtype dtype,
                             const int32_t* tokens, const int32_t* parents,
                             const int32_t* num_nodes, const float* uniforms, int32_t* accept,
                             int32_t* path, int32_t* next_token, int32_t N, int32_t T, int32_t V,
                             void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int dt = enum_code(dtype);
  if (dt != KDA_BF16 && dt != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!verify_sizes_ok(N, T, V)) return KDA_ERR_INVALID_ARG;
  if (N == 0) return KDA_OK;
  if (!target || !tokens || !uniforms || !accept || !path || !next_token) return KDA_ERR_INVALID_ARG;
  if (!aligned16({target, draft}) ||
      !aligned4({tokens, parents, num_nodes, uniforms, accept, path, next_token}))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < kda::verify_workspace(N, T, V))
    return KDA_ERR_WORKSPACE;
  // several workgroups read a sequence's nodes while one writes its results
  const size_t nodes = (size_t)N * T, row = (size_t)V * (dt == KDA_BF16 ? 2 : 4);
  if (!apart({{accept, 4ull * N}, {path, 4 * nodes}, {next_token, 4ull * N}, {workspace, kda::verify_workspace(N, T, V)}},
             {{target, nodes * row}, {draft, nodes * row}, {tokens, 4 * nodes}, {parents, 4 * nodes},
              {num_nodes, 4ull * N}, {uniforms, 4 * nodes}}))
    return KDA_ERR_INVALID_ARG;
  kda::VerifyArgs a;
  a.target = target; a.draft = draft;
  a.tokens = tokens; a.parents = parents; a.num_nodes = num_nodes; a.uniforms = uniforms;
  a.accept = accept; a.path = path; a.next_token = next_token;
  a.N = N; a.T = T; a.V = V;
  a.workspace = workspace;
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_verify(a));
}

namespace {
// Checks and arguments of both directions of the state cache; KDA_OK with
// a->N == 0 when there is nothing to do.
kda_status cache_args(const void* states, const int32_t* slots, const void* values, const uint8_t* scales,
                      int format, int32_t N, int32_t num_slots, int32_t H, int32_t Dk, int32_t Dv,
                      hipStream_t stream, kda::CacheArgs* a) {
  if (format != KDA_CACHE_INT8 && format != KDA_CACHE_E4M3) return KDA_ERR_UNSUPPORTED;
  if (!supported_dims(Dk, Dv)) return KDA_ERR_UNSUPPORTED;
  if (N < 0 || num_slots < 0 || H <= 0 || (int64_t)N * H > kMaxHeads) return KDA_ERR_INVALID_ARG;
  if (!slots && N > num_slots) return KDA_ERR_INVALID_ARG;
  if (N > 0 && (!states || (num_slots > 0 && (!values || !scales)))) return KDA_ERR_INVALID_ARG;
  if (!aligned16({states, values, scales}) || !aligned4({slots})) return KDA_ERR_INVALID_ARG;
  a->states = (float*)states; a->slots = slots;
  a->values = (void*)values; a->scales = (uint8_t*)scales;
  a->N = N; a->num_slots = num_slots; a->H = H; a->D = Dk;
  a->e4m3 = format == KDA_CACHE_E4M3;
  a->stream = stream;
  return KDA_OK;
}
}  // namespace

kda_status kda_state_store(const float* states, const int32_t* slots, void* values,
                           uint8_t* scales, kda_cache_format format, int32_t N,
                           int32_t num_slots, int32_t H, int32_t Dk, int32_t Dv,
                           hipStream_t stream) {
  kda::CacheArgs a;
  const kda_status st =
      cache_args(states, slots, values, scales, enum_code(format), N, num_slots, H, Dk, Dv, stream, &a);
  if (st != KDA_OK || N == 0 || num_slots == 0) return st;
  // (every head reads the slots behind its own)
  if (slots && N > KDA_STORE_MAX_LISTED) return KDA_ERR_INVALID_ARG;
  return from_hip(kda::launch_cache_store(a));
}

kda_status kda_state_load(const void* values, const uint8_t* scales, const int32_t* slots,
                          float* states, kda_cache_format format, int32_t N, int32_t num_slots,
                          int32_t H, int32_t Dk, int32_t Dv, hipStream_t stream) {
  kda::CacheArgs a;
  const kda_status st =
      cache_args(states, slots, values, scales, enum_code(format), N, num_slots, H, Dk, Dv, stream, &a);
  if (st != KDA_OK || N == 0) return st;
  return from_hip(kda::launch_cache_load(a));
}

namespace {

// ---- the layer around a recurrence ----

bool packed_ok(const int32_t* cu, int32_t num_seqs, int32_t T) {
  return T >= 0 && T <= KDA_MAX_PACKED_TOKENS && num_seqs >= 0 && (cu || num_seqs == 1) && aligned4({cu});
}
kda::Packed packed(const int32_t* cu, int32_t num_seqs, int32_t T) { return kda::Packed{cu, num_seqs, T}; }

size_t elem(int dt) { return dt == KDA_BF16 ? 2 : 4; }
// rows of `width` elements, `stride` apart
Span rows(const void* p, int64_t n, int64_t stride, int64_t width, size_t e) {
  return Span{p, n > 0 ? ((size_t)(n - 1) * stride + width) * e : 0};
}
Span flat(const void* p, size_t n, size_t e) { return Span{p, n * e}; }
// A stride holds a row, and the whole array's bytes fit 63 bits.
bool stride_ok(int64_t stride, int64_t width, int64_t n) {
  return stride >= width && stride <= (INT64_MAX / 8 - width) / (n > 0 ? n : 1);
}
bool ssm_size_ok(int32_t N, int32_t P) {
  return (N == 16 || N == 32 || N == 64 || N == 128 || N == 256) && P >= 16 && P <= 256 && P % 16 == 0;
}

kda_status ssm_args(const void* x, int64_t x_stride, const float* dt, const float* a, const void* b,
                    int64_t b_stride, const void* c, int64_t c_stride, const float* skip, const float* dt_bias,
                    int32_t softplus, int dtype, int32_t num_seqs, int32_t T, int32_t H, int32_t G, int32_t N,
                    int32_t P, const float* initial_state, float* final_state, void* y, hipStream_t stream,
                    kda::SsmArgs* out) {
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (!ssm_size_ok(N, P)) return KDA_ERR_UNSUPPORTED;
  if (H <= 0 || G <= 0 || H % G || (softplus != 0 && softplus != 1)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)num_seqs * H > INT32_MAX || (int64_t)T * H > INT32_MAX) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dtype);
  const int64_t xw = (int64_t)H * P, bw = (int64_t)G * N, step = 16 / (int64_t)e;
  if (!stride_ok(x_stride, xw, T) || !stride_ok(b_stride, bw, T) || !stride_ok(c_stride, bw, T) ||
      x_stride > KDA_SSM_MAX_STRIDE || b_stride > KDA_SSM_MAX_STRIDE || c_stride > KDA_SSM_MAX_STRIDE ||
      x_stride % step || b_stride % step || c_stride % step)
    return KDA_ERR_INVALID_ARG;
  if (!a || (T > 0 && (!x || !dt || !b || !c || !y))) return KDA_ERR_INVALID_ARG;
  if (!aligned16({x, dt, a, b, c, skip, dt_bias, initial_state, final_state, y})) return KDA_ERR_INVALID_ARG;
  out->x = x; out->b = b; out->c = c;
  out->x_stride = x_stride; out->b_stride = b_stride; out->c_stride = c_stride;
  out->dt = dt; out->a = a; out->skip = skip; out->dt_bias = dt_bias;
  out->softplus = softplus != 0;
  out->H = H; out->G = G; out->N = N; out->P = P;
  out->initial_state = initial_state; out->final_state = final_state;
  out->y = y;
  out->workspace = nullptr;
  out->bf16 = dtype == KDA_BF16;
  out->stream = stream;
  return KDA_OK;
}

// Whether what a scan writes (y, the state, the workspace) overlaps nothing else.
bool ssm_apart(const kda::SsmArgs& a, int64_t T, int64_t num_seqs, const int32_t* cu, const Span& workspace) {
  const size_t e = a.bf16 ? 2 : 4;
  const Span state = flat(a.final_state, (size_t)num_seqs * a.H * a.N * a.P, 4);
  const Span initial = a.initial_state == a.final_state ? Span{nullptr, 0} : flat(a.initial_state, (size_t)num_seqs * a.H * a.N * a.P, 4);
  return apart({rows(a.y, T, (int64_t)a.H * a.P, (int64_t)a.H * a.P, e), state, workspace},
               {rows(a.x, T, a.x_stride, (int64_t)a.H * a.P, e), rows(a.b, T, a.b_stride, (int64_t)a.G * a.N, e),
                rows(a.c, T, a.c_stride, (int64_t)a.G * a.N, e), flat(a.dt, (size_t)T * a.H, 4), flat(a.a, a.H, 4),
                flat(a.skip, a.H, 4), flat(a.dt_bias, a.H, 4), initial, flat(cu, cu ? (size_t)num_seqs + 1 : 0, 4)});
}

kda_status conv_args(const void* x, int64_t x_stride, const float* weight, const float* bias, int dtype, int64_t rows_,
                     int32_t C, int32_t width, int32_t activation, void* y, hipStream_t stream, kda::ConvArgs* out) {
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (C < 1 || C > KDA_CONV_MAX_CHANNELS || width < 2 || width > KDA_CONV_MAX_WIDTH) return KDA_ERR_INVALID_ARG;
  if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_INVALID_ARG;
  if (!stride_ok(x_stride, C, rows_)) return KDA_ERR_INVALID_ARG;
  if (!weight || (rows_ > 0 && (!x || !y))) return KDA_ERR_INVALID_ARG;
  if (!aligned16({x, weight, bias, y})) return KDA_ERR_INVALID_ARG;
  out->x = x; out->x_stride = x_stride;
  out->weight = weight; out->bias = bias;
  out->C = C; out->width = width;
  out->silu = activation == KDA_ACT_SILU;
  out->y = y;
  out->bf16 = dtype == KDA_BF16;
  out->stream = stream;
  return KDA_OK;
}

// Checks both norms share.
kda_status norm_args_ok(int dtype, int32_t T, int32_t D, int32_t activation, float eps) {
  if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (T < 0 || D < 1 || D > KDA_NORM_MAX || activation < KDA_ACT_NONE || activation > KDA_ACT_SIGMOID)
    return KDA_ERR_INVALID_ARG;
  return eps >= 0.f && eps <= FLT_MAX ? KDA_OK : KDA_ERR_INVALID_ARG;
}

}  // namespace

kda_status kda_conv_prefill(const void* x, int64_t x_stride, const float* weight, const float* bias, kda_dtype dtype,
                            const int32_t* cu_seqlens, int32_t num_seqs, int32_t T, int32_t C, int32_t width,
                            int32_t activation, const void* initial_state, void* final_state, void* y,
                            hipStream_t stream) {
  const int dt = enum_code(dtype);
  kda::ConvArgs a;
  const kda_status st = conv_args(x, x_stride, weight, bias, dt, T, C, width, activation, y, stream, &a);
  if (st != KDA_OK) return st;
  if (!packed_ok(cu_seqlens, num_seqs, T) || !aligned16({initial_state, final_state})) return KDA_ERR_INVALID_ARG;
  a.seqs = packed(cu_seqlens, num_seqs, T);
  a.N = 0;
  a.initial_state = initial_state; a.final_state = final_state;
  if (kda::conv_groups(a) > kda::kMaxConvGroups) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dt), state = (size_t)num_seqs * (width - 1) * C;
  const Span initial = initial_state == final_state ? Span{nullptr, 0} : flat(initial_state, state, e);
  if (!apart({rows(y, T, C, C, e), flat(final_state, state, e)},
             {rows(x, T, x_stride, C, e), flat(weight, (size_t)C * width, 4), flat(bias, C, 4), initial,
              flat(cu_seqlens, cu_seqlens ? (size_t)num_seqs + 1 : 0, 4)}))
    return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  return from_hip(kda::launch_conv(a));
}

kda_status kda_conv_step(const void* x, int64_t x_stride, const float* weight, const float* bias, kda_dtype dtype,
                         void* state, int32_t N, int32_t C, int32_t width, int32_t activation, void* y,
                         hipStream_t stream) {
  const int dt = enum_code(dtype);
  kda::ConvArgs a;
  const kda_status st = conv_args(x, x_stride, weight, bias, dt, N, C, width, activation, y, stream, &a);
  if (st != KDA_OK) return st;
  if (N < 0 || N > KDA_MAX_PACKED_TOKENS || (N > 0 && !state) || !aligned16({state})) return KDA_ERR_INVALID_ARG;
  a.seqs = packed(nullptr, 1, 0);
  a.N = N;
  a.initial_state = state; a.final_state = state;
  const size_t e = elem(dt);
  if (!apart({rows(y, N, C, C, e), flat(state, (size_t)N * (width - 1) * C, e)},
             {rows(x, N, x_stride, C, e), flat(weight, (size_t)C * width, 4), flat(bias, C, 4)}))
    return KDA_ERR_INVALID_ARG;
  if (N == 0) return KDA_OK;
  return from_hip(kda::launch_conv_step(a));
}

size_t kda_ssm_workspace_size(int32_t num_seqs, int32_t T, int32_t H, int32_t N, int32_t P) {
  if (num_seqs < 0 || T < 0 || T > KDA_MAX_PACKED_TOKENS || H <= 0 || (int64_t)T * H > INT32_MAX || !ssm_size_ok(N, P))
    return 0;
  return kda::ssm_workspace(num_seqs, T, H, N, P);
}

kda_status kda_ssm_prefill(const void* x, int64_t x_stride, const float* dt, const float* a, const void* b,
                           int64_t b_stride, const void* c, int64_t c_stride, const float* skip, const float* dt_bias,
                           int32_t dt_softplus, kda_dtype dtype, const int32_t* cu_seqlens, int32_t num_seqs, int32_t T,
                           int32_t H, int32_t G, int32_t N, int32_t P, const float* initial_state, float* final_state,
                           void* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  kda::SsmArgs s;
  if (!packed_ok(cu_seqlens, num_seqs, T)) return KDA_ERR_INVALID_ARG;
  const kda_status st = ssm_args(x, x_stride, dt, a, b, b_stride, c, c_stride, skip, dt_bias, dt_softplus,
                                 enum_code(dtype), num_seqs, T, H, G, N, P, initial_state, final_state, y, stream, &s);
  if (st != KDA_OK) return st;
  s.seqs = packed(cu_seqlens, num_seqs, T);
  if (kda::ssm_threads(s) > kda::kMaxThreads) return KDA_ERR_INVALID_ARG;
  const size_t need = kda::ssm_workspace(num_seqs, T, H, N, P);
  if (need && (!workspace || ((uintptr_t)workspace & 255) || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  s.workspace = workspace;
  if (!ssm_apart(s, T, num_seqs, cu_seqlens, Span{need ? workspace : nullptr, need})) return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  return from_hip(kda::launch_ssm(s));
}

kda_status kda_ssm_step(const void* x, int64_t x_stride, const float* dt, const float* a, const void* b,
                        int64_t b_stride, const void* c, int64_t c_stride, const float* skip, const float* dt_bias,
                        int32_t dt_softplus, kda_dtype dtype, float* state, int32_t num_seqs, int32_t H, int32_t G,
                        int32_t N, int32_t P, void* y, hipStream_t stream) {
  kda::SsmArgs s;
  if (num_seqs < 0 || (num_seqs > 0 && !state)) return KDA_ERR_INVALID_ARG;
  const kda_status st = ssm_args(x, x_stride, dt, a, b, b_stride, c, c_stride, skip, dt_bias, dt_softplus,
                                 enum_code(dtype), num_seqs, num_seqs, H, G, N, P, state, state, y, stream, &s);
  if (st != KDA_OK) return st;
  s.seqs = packed(nullptr, num_seqs, num_seqs);
  if ((int64_t)num_seqs * H * 256 > kda::kMaxThreads) return KDA_ERR_INVALID_ARG;
  if (!ssm_apart(s, num_seqs, num_seqs, nullptr, Span{nullptr, 0})) return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  return from_hip(kda::launch_ssm_step(s));
}

kda_status kda_gated_norm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, const float* weight,
                          int32_t weight_per_head, kda_dtype dtype, int32_t T, int32_t H, int32_t D,
                          int32_t activation, int32_t gate_first, float eps, void* y, hipStream_t stream) {
  const int dt = enum_code(dtype);
  const kda_status st = norm_args_ok(dt, T, D, activation, eps);
  if (st != KDA_OK) return st;
  if (H < 1 || (int64_t)T * H > INT32_MAX || (weight_per_head != 0 && weight_per_head != 1) ||
      (gate_first != 0 && gate_first != 1))
    return KDA_ERR_INVALID_ARG;
  const int64_t w = (int64_t)H * D;
  if (!stride_ok(x_stride, w, T) || (gate && !stride_ok(gate_stride, w, T))) return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (!x || !weight || !y || !aligned16({x, gate, weight, y})) return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dt);
  if (!apart({rows(y, T, w, w, e)}, {rows(x, T, x_stride, w, e), rows(gate, T, gate ? gate_stride : w, w, e),
                                     flat(weight, (weight_per_head ? (size_t)H : 1) * D, 4)}))
    return KDA_ERR_INVALID_ARG;
  kda::GatedNormArgs a;
  a.x = x; a.gate = gate;
  a.x_stride = x_stride; a.gate_stride = gate ? gate_stride : 0;
  a.weight = weight;
  a.T = T; a.H = H; a.D = D; a.act = activation;
  a.weight_per_head = weight_per_head != 0; a.gate_first = gate_first != 0;
  a.eps = eps;
  a.y = y;
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  if (kda::gated_threads(a) > kda::kMaxThreads) return KDA_ERR_INVALID_ARG;
  return from_hip(kda::launch_gated_norm(a));
}

kda_status kda_residual_norm(const void* x, const void* residual, const void* gate, const float* weight,
                             const float* post_weight, const float* scale, kda_dtype dtype, int32_t T, int32_t C,
                             int32_t activation, float alpha, float eps, void* residual_out, void* y,
                             hipStream_t stream) {
  const int dt = enum_code(dtype);
  const kda_status st = norm_args_ok(dt, T, C, activation, eps);
  if (st != KDA_OK) return st;
  if (!(alpha >= -FLT_MAX && alpha <= FLT_MAX)) return KDA_ERR_INVALID_ARG;
  if (T == 0) return KDA_OK;
  if (!x || !weight || !y || !aligned16({x, residual, gate, weight, post_weight, scale, residual_out, y}))
    return KDA_ERR_INVALID_ARG;
  const size_t e = elem(dt), n = (size_t)T * C;
  const Span before = residual == residual_out ? Span{nullptr, 0} : flat(residual, n, e);
  if (!apart({flat(y, n, e), flat(residual_out, n, e)},
             {flat(x, n, e), before, flat(gate, n, e), flat(weight, C, 4), flat(post_weight, C, 4), flat(scale, C, 4)}))
    return KDA_ERR_INVALID_ARG;
  kda::ResidualNormArgs a;
  a.x = x; a.residual = residual; a.gate = gate;
  a.weight = weight; a.post_weight = post_weight; a.scale = scale;
  a.T = T; a.C = C; a.act = activation;
  a.alpha = alpha; a.eps = eps;
  a.residual_out = residual_out; a.y = y;
  a.bf16 = dt == KDA_BF16;
  a.stream = stream;
  return from_hip(kda::launch_residual_norm(a));
}

}  // extern "C"
