"""Thin ctypes binding of libkda (include/kda.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libkda.so. PyTorch supplies device memory and the current stream.
The library must be built (``python -m gated_delta_rule_109_amd.build`` or
``__graft_entry__.build()``); there is no fallback of any kind when it is
missing.
"""
import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# the built library (KDA_LIB names another build of it, e.g. the host-sanitizer one)
LIB_PATH = os.environ.get("KDA_LIB") or os.path.join(HERE, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_HIP = range(5)
KDA_BF16, KDA_F32 = 0, 1
CHUNK = 16
LN_HALF = math.log(0.5)

EXPORTED = ("kda_status_string", "kda_prefill_num_checkpoints", "kda_prefill_workspace_size",
            "kda_prefill_workspace_size_window", "kda_prefill_chunked", "kda_prefill_chunked_ex", "kda_prefill_chunked_noalloc",
            "kda_decode_step", "kda_decode_tokens", "kda_decode_tree", "kda_commit_path",
            "kda_verify_workspace_size", "kda_verify_drafts", "kda_state_store", "kda_state_load")
DECODE_MAX_TOKENS = 16
TREE_MAX_NODES = 64
CACHE_INT8, CACHE_E4M3 = 0, 1
INT32_MAX = 2 ** 31 - 1
CACHE_BLOCK = 32                                 # values that share a scale
FE_L2NORM_QK, FE_GATE_LOGITS, FE_BETA_LOGITS = 1, 2, 4
FE_ALL = FE_L2NORM_QK | FE_GATE_LOGITS | FE_BETA_LOGITS
GATE_CHANNEL, GATE_HEAD, GATE_NONE = 0, 1, 2     # KDA, Gated DeltaNet, DeltaNet


MAX_SEGMENTS = 16
SEGMENT_SLICE_LIMIT = 80          # forced segments need num_seqs * H * (D / 16) <= this
NOALLOC_SCRATCH_BYTES = 256 << 20  # static scratch of kda_prefill_chunked_noalloc


class Options(ctypes.Structure):
    """kda_options: which inputs are raw (FE_* flags), the norm epsilon, the
    gate layout (GATE_CHANNEL: g [.., H, D]; GATE_HEAD: g [.., H]; GATE_NONE:
    no g), and the prefill's segments per sequence (0: the library's choice,
    1: none, 2 .. MAX_SEGMENTS: forced)."""
    _fields_ = [("flags", ctypes.c_uint32), ("norm_eps", ctypes.c_float), ("gate", ctypes.c_int32),
                ("segments", ctypes.c_int32)]

    def __init__(self, flags=0, norm_eps=1e-6, gate=GATE_CHANNEL, segments=0):
        super().__init__(int(flags), float(norm_eps), int(gate), int(segments))

_lib = None
_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i32p = ctypes.POINTER(ctypes.c_int32)


class KdaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {lib().kda_status_string(status).decode()}")


def lib():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.kda_status_string.restype = ctypes.c_char_p
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_prefill_num_checkpoints.restype = ctypes.c_int64
        L.kda_prefill_num_checkpoints.argtypes = [_i32p, _i32, _i32]
        L.kda_prefill_workspace_size.restype = ctypes.c_size_t
        L.kda_prefill_workspace_size.argtypes = [_i32, ctypes.c_int64, _i32, _i32, _i32]
        L.kda_prefill_workspace_size_window.restype = ctypes.c_size_t
        L.kda_prefill_workspace_size_window.argtypes = [_i32, ctypes.c_int64, _i32, _i32, _i32, ctypes.c_int64]
        L.kda_prefill_chunked.restype = ctypes.c_int
        L.kda_prefill_chunked.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _i32p, _i32,
                                          _i32, _i32, _i32, ctypes.c_float, ctypes.c_float, _vp,
                                          _vp, _i32, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.kda_decode_step.restype = ctypes.c_int
        L.kda_decode_step.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _i32, _i32,
                                      _i32, _i32, ctypes.c_float, ctypes.c_float, _vp]
        L.kda_decode_tokens.restype = ctypes.c_int
        L.kda_decode_tokens.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i32,
                                        _i32, _i32, _i32, _i32, ctypes.c_float, ctypes.c_float,
                                        ctypes.POINTER(Options), _vp]
        L.kda_prefill_chunked_ex.restype = ctypes.c_int
        L.kda_prefill_chunked_ex.argtypes = L.kda_prefill_chunked.argtypes[:-1] + [
            ctypes.POINTER(Options), _vp]
        L.kda_prefill_chunked_noalloc.restype = ctypes.c_int
        L.kda_prefill_chunked_noalloc.argtypes = L.kda_prefill_chunked.argtypes[:-3] + [
            ctypes.POINTER(Options), _vp]
        L.kda_decode_tree.restype = ctypes.c_int
        L.kda_decode_tree.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                      _i32, _i32, ctypes.c_float, ctypes.c_float, ctypes.POINTER(Options), _vp]
        L.kda_commit_path.restype = ctypes.c_int
        L.kda_commit_path.argtypes = [_vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                                      ctypes.c_float, ctypes.POINTER(Options), _vp]
        L.kda_verify_workspace_size.restype = ctypes.c_size_t
        L.kda_verify_workspace_size.argtypes = [_i32, _i32, _i32]
        L.kda_verify_drafts.restype = ctypes.c_int
        L.kda_verify_drafts.argtypes = [_vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32,
                                        _vp, ctypes.c_size_t, _vp]
        L.kda_state_store.restype = ctypes.c_int
        L.kda_state_store.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, _i32, _i32, _i32, _i32, _i32, _vp]
        L.kda_state_load.restype = ctypes.c_int
        L.kda_state_load.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int, _i32, _i32, _i32, _i32, _i32, _vp]
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _host_cu(cu_seqlens):
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int32).cpu().contiguous()
    return cu, cu.numpy().ctypes.data_as(_i32p)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous device tensors")


def _expect(t, name, shape, dtype):
    """The C ABI takes raw pointers and cannot see sizes: a wrong shape would
    make a kernel read or write out of bounds, so every tensor is checked here
    before any call."""
    if t is None:
        return
    if t.shape != shape:      # torch.Size compares as the tuple it is
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")


def _gate_shape(lead, H, D, options):
    """Shape of g for the gate layout of `options` (None: no g is read)."""
    gate = GATE_CHANNEL if options is None else options.gate
    if gate == GATE_NONE:
        return None
    return (*lead, H, D) if gate == GATE_CHANNEL else (*lead, H)


def _check_inputs(q, k, v, g, beta, lead, H, D, options, beta_shape):
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q/k/v must be bfloat16 or float32, got {q.dtype}")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _expect(t, name, (*lead, H, D), q.dtype)
    gshape = _gate_shape(lead, H, D, options)
    if gshape is None:
        g = None
    elif g is None:
        raise ValueError("g is required by this gate layout")
    _expect(g, "g", gshape if gshape else (), torch.float32)
    _expect(beta, "beta", beta_shape, torch.float32)
    return g


def num_checkpoints(cu_seqlens, ckpt_interval: int) -> int:
    cu, p = _host_cu(cu_seqlens)
    r = lib().kda_prefill_num_checkpoints(p, len(cu) - 1, int(ckpt_interval))
    if r < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefill_num_checkpoints")
    return int(r)


def kda_check_cu(cu_host) -> int:
    """-1 if the host offsets are malformed (cu[0] != 0 or decreasing)."""
    return lib().kda_prefill_num_checkpoints(cu_host.numpy().ctypes.data_as(_i32p), len(cu_host) - 1, 0)


def workspace_size(num_seqs: int, total_tokens: int, H: int, D: int,
                   window_blocks: Optional[int] = None) -> int:
    """kda_prefill_workspace_size: bytes of device workspace for num_seqs
    sequences of total_tokens packed tokens (independent of the lengths);
    with window_blocks, kda_prefill_workspace_size_window: the bytes that run
    the call with the records of at most that many 32-token blocks at a time."""
    if window_blocks is None:
        return int(lib().kda_prefill_workspace_size(int(num_seqs), int(total_tokens), H, D, D))
    return int(lib().kda_prefill_workspace_size_window(int(num_seqs), int(total_tokens), H, D, D,
                                                       int(window_blocks)))


@dataclass
class PrefillPlan:
    """Host and device copies of cu_seqlens plus a workspace sized for them
    (None for kda_prefill_chunked_noalloc, which uses the library's static
    scratch)."""
    cu_host: torch.Tensor
    cu_dev: torch.Tensor
    workspace: Optional[torch.Tensor]
    num_ckpt: int
    ckpt_interval: int


def make_plan(cu_seqlens, H: int, D: int, device, ckpt_interval: int = 0,
              workspace: bool = True, window_blocks: Optional[int] = None) -> PrefillPlan:
    """window_blocks: size the workspace for record windows of at most that
    many blocks (None: the library's default size)."""
    cu_host, p = _host_cu(cu_seqlens)
    if int(kda_check_cu(cu_host)) < 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "cu_seqlens")
    if workspace:
        ws = workspace_size(len(cu_host) - 1, int(cu_host[-1]), H, D, window_blocks)
        if ws == 0:
            raise KdaError(KDA_ERR_INVALID_ARG, "kda_prefill_workspace_size")
        workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=device)
    else:
        workspace = None
    return PrefillPlan(cu_host, cu_host.to(device), workspace,
                       num_checkpoints(cu_host, ckpt_interval) if ckpt_interval else 0,
                       int(ckpt_interval))


def _opt_ptr(options: Optional[Options]):
    return None if options is None else ctypes.byref(options)


def prefill(q, k, v, g, beta, cu_seqlens=None, initial_state=None, scale=1.0, g_min=LN_HALF,
            ckpt_interval=0, out_final_state=True, plan: Optional[PrefillPlan] = None,
            o=None, final_state=None, checkpoints=None, options: Optional[Options] = None,
            noalloc: bool = False):
    """kda_prefill_chunked on packed [T, H, D] tensors (kda_prefill_chunked_ex
    when Options are given: gate layout, and q, k, g, beta raw as the flags
    say; kda_prefill_chunked_noalloc when noalloc is set: no workspace, the
    library's static scratch instead).

    Returns (o, final_state or None, checkpoints or None)."""
    T, H, D = q.shape
    if plan is None:
        plan = make_plan([0, T] if cu_seqlens is None else cu_seqlens, H, D, q.device, ckpt_interval,
                         workspace=not noalloc)
    N = len(plan.cu_host) - 1
    if int(plan.cu_host[-1]) != T:
        raise ValueError(f"cu_seqlens ends at {int(plan.cu_host[-1])}, but q holds {T} tokens")
    g = _check_inputs(q, k, v, g, beta, (T,), H, D, options, (T, H))
    _expect(initial_state, "initial_state", (N, H, D, D), torch.float32)
    _expect(o, "o", (T, H, D), q.dtype)
    _expect(final_state, "final_state", (N, H, D, D), torch.float32)
    _expect(checkpoints, "checkpoints", (plan.num_ckpt, H, D, D), torch.float32)
    _check_dev(q, k, v, g, beta, initial_state, o, final_state, checkpoints)
    if o is None:
        o = torch.empty_like(v)
    if final_state is None and out_final_state:
        final_state = torch.empty(N, H, D, D, dtype=torch.float32, device=q.device)
    if checkpoints is None and plan.num_ckpt > 0:
        checkpoints = torch.empty(plan.num_ckpt, H, D, D, dtype=torch.float32, device=q.device)
    args = (_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(g), _ptr(beta), _ptr(plan.cu_dev),
            plan.cu_host.numpy().ctypes.data_as(_i32p), N, H, D, v.shape[2], float(scale),
            float(g_min), _ptr(initial_state), _ptr(final_state), plan.ckpt_interval,
            _ptr(checkpoints), _ptr(o))
    if noalloc:
        st = lib().kda_prefill_chunked_noalloc(*args, _opt_ptr(options), _stream(q.device))
        if st != KDA_OK:
            raise KdaError(st, "kda_prefill_chunked_noalloc")
        return o, final_state, checkpoints
    if plan.workspace is None:
        raise ValueError("this plan has no workspace (made for the noalloc entry point)")
    args += (_ptr(plan.workspace), plan.workspace.numel())
    if options is None:
        st = lib().kda_prefill_chunked(*args, _stream(q.device))
    else:
        st = lib().kda_prefill_chunked_ex(*args, _opt_ptr(options), _stream(q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_prefill_chunked")
    return o, final_state, checkpoints


def decode_step(q, k, v, g, beta, state, scale=1.0, g_min=LN_HALF, o=None):
    """kda_decode_step: q,k,g [N,H,D]; v [N,H,D]; beta [N,H]; state [N,H,D,D]
    updated in place. Returns o [N,H,D]."""
    N, H, D = q.shape
    _check_inputs(q, k, v, g, beta, (N,), H, D, None, (N, H))
    _expect(state, "state", (N, H, D, D), torch.float32)
    _expect(o, "o", (N, H, D), q.dtype)
    _check_dev(q, k, v, g, beta, state, o)
    if o is None:
        o = torch.empty_like(v)
    st = lib().kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(g), _ptr(beta),
                               _ptr(state), _ptr(o), N, H, D, v.shape[2], float(scale),
                               float(g_min), _stream(q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step")
    return o


def decode_tokens(q, k, v, g, beta, state, accept=None, scale=1.0, g_min=LN_HALF, o=None,
                  options: Optional[Options] = None):
    """kda_decode_tokens: q,k,g,v [N,T,H,D]; beta [N,T,H]; state [N,H,D,D]
    updated in place to the state after accept[n] tokens (all T when accept is
    None); accept is a device int32 [N] tensor; options as in prefill.
    Returns o [N,T,H,D]."""
    N, T, H, D = q.shape
    g = _check_inputs(q, k, v, g, beta, (N, T), H, D, options, (N, T, H))
    _expect(state, "state", (N, H, D, D), torch.float32)
    _expect(accept, "accept", (N,), torch.int32)
    _expect(o, "o", (N, T, H, D), q.dtype)
    _check_dev(q, k, v, g, beta, state, accept, o)
    if o is None:
        o = torch.empty_like(v)
    st = lib().kda_decode_tokens(_ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(g), _ptr(beta),
                                 _ptr(state), _ptr(accept), _ptr(o), N, T, H, D, v.shape[3],
                                 float(scale), float(g_min), _opt_ptr(options), _stream(q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_tokens")
    return o


# ---- one speculative step over trees of drafted tokens ---------------------------

def _check_step(*specs):
    """Every given tensor (name, tensor or None, shape, dtype; the first one not
    None) has its shape and dtype, is contiguous, and all are on one device,
    whose index is returned. One pass over what is right; the first thing wrong
    is looked up after it."""
    dev = specs[0][1].get_device()
    for _, t, shape, dtype in specs:
        if t is not None and (t.shape != shape or t.dtype is not dtype or not t.is_contiguous()
                              or t.get_device() != dev):
            break
    else:
        if dev >= 0:
            return dev
    for name, t, shape, dtype in specs:
        _expect(t, name, shape, dtype)
    _check_dev(*(t for _, t, _, _ in specs))
    raise ValueError("tensors on more than one device: one call takes one device")


def _check_int32(a, b, c):
    """Sizes that the C ABI's int32 cannot carry (ctypes would drop the high bits)."""
    if a > INT32_MAX or b > INT32_MAX or c > INT32_MAX:
        raise ValueError(f"sizes {a}, {b}, {c}: one is outside int32")


def _step_inputs(q, k, v, g, beta, lead, H, D, options):
    """Specifications of a step's q, k, v, g and beta."""
    dt = q.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise TypeError(f"q/k/v must be bfloat16 or float32, got {dt}")
    _check_int32(lead[0], lead[1], H)
    shape = (*lead, H, D)
    gshape = _gate_shape(lead, H, D, options)
    if gshape is None:
        g = None
    elif g is None:
        raise ValueError("g is required by this gate layout")
    return (("q", q, shape, dt), ("k", k, shape, dt), ("v", v, shape, dt), ("g", g, gshape, torch.float32),
            ("beta", beta, (*lead, H), torch.float32)), g


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(dev, where, fn, *args):
    """fn(*args, stream) on device dev's current stream, with dev current. These
    calls take microseconds, so device and stream are read as the numbers they
    are (a torch.cuda.Stream around the handle costs 2.2 us of a call's 13)."""
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(dev, where, fn, *args)
    st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != KDA_OK:
        raise KdaError(st, where)


def decode_tree(q, k, v, g, beta, state, parents=None, num_nodes=None, scale=1.0, g_min=LN_HALF, o=None,
                options: Optional[Options] = None):
    """kda_decode_tree: the outputs of T drafted tokens per sequence that form
    a tree (parents, device int32 [N,T]; None: a chain), each over the state
    [N,H,D,D] and its own path; the state is only read. q,k,g,v [N,T,H,D] and
    beta [N,T,H] as in decode_tokens; num_nodes (device int32 [N]) gives each
    sequence its own number of nodes, whose other rows of o stay as they are.
    Returns o [N,T,H,D]."""
    N, T, H, D = q.shape
    specs, g = _step_inputs(q, k, v, g, beta, (N, T), H, D, options)
    dev = _check_step(*specs, ("state", state, (N, H, D, D), torch.float32),
                      ("parents", parents, (N, T), torch.int32), ("num_nodes", num_nodes, (N,), torch.int32),
                      ("o", o, (N, T, H, D), q.dtype))
    if o is None:
        o = torch.empty_like(v) if num_nodes is None else torch.zeros_like(v)
    _call(dev, "kda_decode_tree", lib().kda_decode_tree, q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q),
          _addr(g), _addr(beta), _addr(state), _addr(parents), _addr(num_nodes), o.data_ptr(), N, T, H, D, D,
          float(scale), float(g_min), _opt_ptr(options))
    return o


def commit_path(k, v, g, beta, state, path, accept, g_min=LN_HALF, options: Optional[Options] = None):
    """kda_commit_path: the recurrence over nodes path[n, :accept[n]] (device
    int32 [N,T] and [N], as verify_drafts returns them) on state [N,H,D,D], in
    place; k, v, g, beta and options are those of decode_tree. Returns state."""
    N, T, H, D = k.shape
    if path is None or accept is None:
        raise ValueError("path and accept are required")
    specs, g = _step_inputs(k, k, v, g, beta, (N, T), H, D, options)
    dev = _check_step(*specs[1:], ("state", state, (N, H, D, D), torch.float32), ("path", path, (N, T), torch.int32),
                      ("accept", accept, (N,), torch.int32))
    _call(dev, "kda_commit_path", lib().kda_commit_path, k.data_ptr(), v.data_ptr(), _dtype_code(k), _addr(g),
          _addr(beta), _addr(state), path.data_ptr(), accept.data_ptr(), N, T, H, D, D, float(g_min),
          _opt_ptr(options))
    return state


def verify_workspace(N: int, T: int, V: int, device) -> torch.Tensor:
    """A workspace for verify_drafts calls of these sizes and smaller ones, one
    after another."""
    _check_int32(N, T, V)
    size = int(lib().kda_verify_workspace_size(int(N), int(T), int(V)))
    if size == 0 and N != 0:
        raise KdaError(KDA_ERR_INVALID_ARG, "kda_verify_workspace_size")
    return torch.empty(max(size, 256), dtype=torch.uint8, device=device)


def verify_drafts(target, draft, tokens, uniforms, parents=None, num_nodes=None,
                  workspace: Optional[torch.Tensor] = None, accept=None, path=None, next_token=None):
    """kda_verify_drafts: rejection sampling of drafted tokens, without loss for
    rows that sum to 1 (rows are never normalised; what bfloat16 rows shift is
    in kda.h). target [N,T,V] (bfloat16 or float32) holds the target's probabilities after each node,
    draft [N,T,V] those that a node's children were drawn from (None: chosen
    without sampling); tokens int32 [N,T]; uniforms float32 [N,T], entry i >= 1
    for node i's test and entry 0 for the next token; parents and num_nodes as
    in decode_tree. workspace (verify_workspace) is allocated when None, and so
    are the outputs, which must not overlap each other or an input.
    Returns (accept [N], path [N,T], next_token [N]), int32: accept is that of
    decode_tokens (chains) and, with path, of commit_path."""
    N, T, V = target.shape
    _check_int32(N, T, V)
    code = _dtype_code(target)
    if tokens is None or uniforms is None:
        raise ValueError("tokens and uniforms are required")
    i32 = torch.int32
    dev = _check_step(("target", target, (N, T, V), target.dtype), ("draft", draft, (N, T, V), target.dtype),
                      ("tokens", tokens, (N, T), i32), ("uniforms", uniforms, (N, T), torch.float32),
                      ("parents", parents, (N, T), i32), ("num_nodes", num_nodes, (N,), i32),
                      ("workspace", workspace, None if workspace is None else (workspace.numel(),), torch.uint8),
                      ("accept", accept, (N,), i32), ("path", path, (N, T), i32), ("next_token", next_token, (N,), i32))
    if workspace is None:
        workspace = verify_workspace(N, T, V, target.device)
    if accept is None:
        accept = tokens.new_empty(N)
    if path is None:
        path = torch.empty_like(tokens)
    if next_token is None:
        next_token = tokens.new_empty(N)
    _call(dev, "kda_verify_drafts", lib().kda_verify_drafts, target.data_ptr(), _addr(draft), code, tokens.data_ptr(),
          _addr(parents), _addr(num_nodes), uniforms.data_ptr(), accept.data_ptr(), path.data_ptr(),
          next_token.data_ptr(), N, T, V, workspace.data_ptr(), workspace.numel())
    return accept, path, next_token


# ---- 8-bit cache of recurrent states -----------------------------------------------

@dataclass
class StateCache:
    """values [num_slots,H,D,D] (int8, or float8_e4m3fn) and scales
    [num_slots,H,D*D/32] (uint8: the step's exponent + 127)."""
    values: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        if self.values.dtype not in (torch.int8, torch.float8_e4m3fn):
            raise TypeError(f"values: expected torch.int8 or torch.float8_e4m3fn, got {self.values.dtype}")
        if self.values.dim() != 4 or self.values.shape[2] != self.values.shape[3]:
            raise ValueError(f"values: expected shape [num_slots, H, D, D], got {tuple(self.values.shape)}")
        S, H, D, _ = self.values.shape
        _expect(self.scales, "scales", (S, H, D * D // CACHE_BLOCK), torch.uint8)

    @property
    def format(self) -> int:
        return CACHE_INT8 if self.values.dtype == torch.int8 else CACHE_E4M3


def make_state_cache(num_slots: int, H: int, D: int, device, dtype=torch.int8) -> StateCache:
    """A cache of num_slots states, every slot the zero state."""
    return StateCache(torch.zeros(num_slots, H, D, D, dtype=dtype, device=device),
                      torch.zeros(num_slots, H, D * D // CACHE_BLOCK, dtype=torch.uint8, device=device))


def _cache_call(where, fn, first, cache: StateCache, slots, states):
    S, H, D, _ = cache.values.shape
    N = states.shape[0]
    dev = _check_step(("values", cache.values, (S, H, D, D), cache.values.dtype),
                      ("scales", cache.scales, (S, H, D * D // CACHE_BLOCK), torch.uint8),
                      ("slots", slots, (N,), torch.int32), ("states", states, (N, H, D, D), torch.float32))
    _check_int32(S, N, H)
    if first == "states":
        args = (states.data_ptr(), _addr(slots), cache.values.data_ptr(), cache.scales.data_ptr())
    else:
        args = (cache.values.data_ptr(), cache.scales.data_ptr(), _addr(slots), states.data_ptr())
    _call(dev, where, fn, *args, cache.format, N, S, H, D, D)


def state_store(states, cache: StateCache, slots=None):
    """kda_state_store: states [N,H,D,D] into the cache's slots (device int32
    [N]; None: slot n), quantised to 8 bits. A state whose slot is outside the
    cache is not written; of two states for one slot the later one is. With
    slots the time grows with H N^2 (see kda.h)."""
    _cache_call("kda_state_store", lib().kda_state_store, "states", cache, slots, states)


def state_load(cache: StateCache, slots=None, states=None):
    """kda_state_load: the states of the given slots (None: all), float32
    [N,H,D,D]; a slot outside the cache reads as the zero state."""
    if states is None:
        N = cache.values.shape[0] if slots is None else slots.shape[0]
        states = torch.empty(N, *cache.values.shape[1:], dtype=torch.float32, device=cache.values.device)
    _cache_call("kda_state_load", lib().kda_state_load, "cache", cache, slots, states)
    return states
