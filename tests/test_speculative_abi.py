"""Refusals of the speculative step and the state cache, through the C ABI and
through the binding (no GPU: everything here is refused before device work, or
there is nothing to do), and the C ABI part again with the host code built
under AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from gated_delta_rule_109_amd import kda, profiling

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)             # a 16- and 256-byte aligned address that is never read
ODD = ctypes.c_void_p(4100)           # 4-byte aligned: enough for int32 arrays and uniforms only
ODD2 = ctypes.c_void_p(4098)
OK, BAD, UNSUP, WS = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
INT_MAX = 2 ** 31 - 1


def opt(**k):
    return ctypes.byref(kda.Options(**k))


def tree(**k):
    a = dict(q=P, k=P, v=P, dtype=0, g=P, beta=P, state=P, parents=P, num_nodes=P, o=P, N=2, T=5, H=3, Dk=128, Dv=128,
             scale=1.0, g_min=-0.5, opt=None, stream=None)
    assert set(k) <= set(a)
    a.update(k)
    return kda.lib().kda_decode_tree(*a.values())


def commit(**k):
    a = dict(k=P, v=P, dtype=0, g=P, beta=P, state=P, path=P, accept=P, N=2, T=5, H=3, Dk=128, Dv=128, g_min=-0.5,
             opt=None, stream=None)
    assert set(k) <= set(a)
    a.update(k)
    return kda.lib().kda_commit_path(*a.values())


def verify(**k):
    a = dict(target=P, draft=P, dtype=1, tokens=P, parents=P, num_nodes=P, uniforms=P, accept=P, path=P, next_token=P,
             N=2, T=5, V=1000, workspace=P, workspace_bytes=1 << 30, stream=None)
    assert set(k) <= set(a)
    a.update(k)
    return kda.lib().kda_verify_drafts(*a.values())


def store(**k):
    a = dict(states=P, slots=P, values=P, scales=P, format=0, N=2, num_slots=4, H=3, Dk=128, Dv=128, stream=None)
    assert set(k) <= set(a)
    a.update(k)
    return kda.lib().kda_state_store(*a.values())


def load(**k):
    a = dict(values=P, scales=P, slots=P, states=P, format=0, N=2, num_slots=4, H=3, Dk=128, Dv=128, stream=None)
    assert set(k) <= set(a)
    a.update(k)
    return kda.lib().kda_state_load(*a.values())


@pytest.mark.parametrize("call", [tree, commit])
@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), UNSUP), (dict(Dk=64, Dv=64), UNSUP), (dict(Dv=16), UNSUP), (dict(T=0), BAD),
    (dict(T=kda.TREE_MAX_NODES + 1), BAD), (dict(N=-1), BAD), (dict(H=0), BAD), (dict(g_min=0.1), BAD),
    (dict(g_min=float("nan")), BAD), (dict(g_min=float("-inf")), BAD), (dict(N=INT_MAX), BAD),
    (dict(N=1 << 20, H=1 << 10), BAD),
    (dict(N=1 << 20, H=16, T=1), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(g=None), BAD),
    (dict(beta=None), BAD), (dict(state=None), BAD), (dict(k=ODD), BAD), (dict(state=ODD), BAD),
])
def test_tree_and_commit_refuse(call, bad, status):
    assert call(**bad) == status


@pytest.mark.parametrize("call", [tree, commit])
def test_tree_and_commit_options(call):
    assert call(opt=opt(flags=8)) == BAD
    assert call(opt=opt(gate=3)) == BAD
    assert call(opt=opt(flags=kda.FE_GATE_LOGITS, gate=kda.GATE_NONE)) == BAD
    assert call(opt=opt(norm_eps=-1.0)) == BAD
    assert call(opt=opt(gate=kda.GATE_NONE), g=None, state=None) == BAD     # g is not what is missing
    assert call(N=0, k=None, v=None) == OK


def test_tree_launch_limits():
    """Trees of more than 16 nodes with heads of 128 launch 512 threads a head:
    a launch of 2^32 threads or more is refused before it is tried."""
    assert tree(N=1 << 18, H=32, T=17) == BAD                 # 2^23 heads: 2^32 threads
    assert tree(N=1 << 18, H=32, T=64) == BAD


def test_tree_and_commit_own_pointers():
    for name in ("q", "o"):
        assert tree(**{name: None}) == BAD and tree(**{name: ODD}) == BAD
    for name in ("parents", "num_nodes"):
        assert tree(**{name: ODD2}) == BAD and tree(**{name: ODD}, q=None) == BAD
    for name in ("path", "accept"):
        assert commit(**{name: None}) == BAD and commit(**{name: ODD2}) == BAD


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), UNSUP), (dict(N=-1), BAD), (dict(T=0), BAD), (dict(T=65), BAD), (dict(V=0), BAD), (dict(V=(1 << 24) + 1), BAD),
    (dict(N=1 << 20, T=1), BAD), (dict(target=None), BAD), (dict(tokens=None), BAD), (dict(uniforms=None), BAD),
    (dict(accept=None), BAD), (dict(path=None), BAD), (dict(next_token=None), BAD), (dict(target=ODD), BAD),
    (dict(draft=ODD), BAD), (dict(parents=ODD2), BAD), (dict(uniforms=ODD2), BAD), (dict(tokens=ODD, workspace=None), WS), (dict(workspace=None), WS), (dict(workspace=ctypes.c_void_p(4112)), WS),
    (dict(workspace_bytes=0), WS), (dict(N=0, target=None, workspace=None), OK),
])
def test_verify_refuses(bad, status):
    assert verify(**bad) == status


# every array of a verification 1 MiB from the next, so that none overlaps
APART = {name: (1 << 20) * (i + 1) for i, name in enumerate(
    ("target", "draft", "tokens", "parents", "num_nodes", "uniforms", "accept", "path", "next_token", "workspace"))}


@pytest.mark.parametrize("out", ["accept", "path", "next_token", "workspace"])
@pytest.mark.parametrize("other", list(APART))
def test_verify_refuses_outputs_that_overlap(out, other):
    """An output on top of another array, or with its first or last bytes in it:
    workgroups read a sequence's nodes while one of them writes."""
    if out == other:
        return
    N, T, V = 2, 5, 1000
    bytes_of = dict(target=4 * N * T * V, draft=4 * N * T * V, tokens=4 * N * T, parents=4 * N * T, num_nodes=4 * N,
                    uniforms=4 * N * T, accept=4 * N, path=4 * N * T, next_token=4 * N,
                    workspace=kda.lib().kda_verify_workspace_size(N, T, V))
    step = 256 if out == "workspace" else 4
    for at in (0, bytes_of[other] - 1 & -step, -(bytes_of[out] - 1 & -step)):
        a = {**APART, out: APART[other] + at}
        assert verify(**{k: ctypes.c_void_p(x) for k, x in a.items()}, N=N, T=T, V=V) == BAD


def test_verify_workspace_size():
    size = kda.lib().kda_verify_workspace_size
    assert size(0, 5, 100) == 0 and size(-1, 5, 100) == 0 and size(1, 0, 100) == 0 and size(1, 65, 100) == 0
    assert size(1, 5, 0) == 0 and size(1, 5, (1 << 24) + 1) == 0 and size(1 << 20, 2, 10) == 0 and size((1 << 20) - 1, 2, 10) > 0
    for N, V in ((1, 1), (1, 32768), (256, 131072), (63, 50001), (64, 50001), (3, 1 << 24)):
        s = size(N, 5, V)
        assert N * 32 <= s <= 1024 * N + 512 + 16 * N and s % 256 == 0
        assert verify(N=N, V=V, workspace_bytes=s - 1) == WS


def test_verify_workspace_serves_smaller_calls():
    """A server allocates once for its largest sizes: no smaller batch, tree or
    vocabulary needs more."""
    size = kda.lib().kda_verify_workspace_size
    some_n = [1, 2, 16, 17, 31, 48, 62, 63, 64, 65, 66, 96, 128, 200, 255, 256, 257, 300, 512, 1000, 4096, 1 << 16, (1 << 20) - 1]
    some_v = [1, 7, 1000, 1024, 1025, 4096, 4097, 32768, 50001, 65535, 65536, 65537, 66048, 66049, 131072, 262144, 262145,
              300001, 1 << 20, 2000003, (1 << 24) - 1, 1 << 24]
    for V in some_v:
        sizes = [size(N, 5, V) for N in some_n]
        assert sizes == sorted(sizes), V
        assert size(64, 1, V) == size(64, 64, V)
    for N in some_n:
        sizes = [size(N, 5, V) for V in some_v]
        assert sizes == sorted(sizes), N
        sizes = [size(N, 5, V) for V in range(60000, 70000, 7)]
        assert sizes == sorted(sizes), N
    for V in (32768, 50001, 65536, 131072):
        sizes = [size(N, 5, V) for N in range(0, 300)]
        assert sizes == sorted(sizes), V


@pytest.mark.parametrize("call", [store, load])
@pytest.mark.parametrize("bad,status", [
    (dict(format=2), UNSUP), (dict(format=-1), UNSUP), (dict(Dk=64, Dv=64), UNSUP), (dict(Dv=16), UNSUP),
    (dict(N=-1), BAD), (dict(num_slots=-1), BAD), (dict(H=0), BAD), (dict(N=1 << 20, H=16), BAD),
    (dict(slots=None, N=5), BAD), (dict(states=None), BAD), (dict(values=None), BAD), (dict(scales=None), BAD),
    (dict(states=ODD), BAD), (dict(slots=ODD2), BAD), (dict(values=ODD), BAD), (dict(scales=ODD), BAD),
    (dict(N=0, states=None, values=None, scales=None), OK),
])
def test_cache_refuses(call, bad, status):
    assert call(**bad) == status


def test_store_refuses_longer_lists():
    assert store(N=(1 << 20) + 1, H=1) == BAD
    assert store(N=(1 << 20) + 1, H=1, num_slots=0) == OK      # nothing to store into


def test_nothing_to_store_into():
    assert store(num_slots=0, values=None, scales=None) == OK


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


I32, BF16 = torch.int32, torch.bfloat16


def test_binding_checks_tree_and_commit():
    x = t(3, 5, 2, 16, dtype=BF16)
    ok = dict(q=x, k=x, v=x, g=t(3, 5, 2, 16), beta=t(3, 5, 2), state=t(3, 2, 16, 16))
    for name, bad, err, msg in (
            ("k", t(3, 5, 2, 8, dtype=BF16), ValueError, "k: expected shape"), ("g", t(3, 5, 2), ValueError, "g: expected"),
            ("state", t(2, 2, 16, 16), ValueError, "state: expected shape"),
            ("state", t(3, 2, 16, 16, dtype=BF16), TypeError, "state: expected"),
            ("parents", t(3, 4, dtype=I32), ValueError, "parents: expected shape"),
            ("parents", t(3, 5), TypeError, "parents: expected torch.int32"),
            ("num_nodes", t(3, 1, dtype=I32), ValueError, "num_nodes: expected shape"),
            ("o", t(3, 5, 2, 16), TypeError, "o: expected")):
        with pytest.raises(err, match=msg):
            kda.decode_tree(**{**ok, name: bad})
    with pytest.raises(ValueError, match="contiguous device tensors"):
        kda.decode_tree(**ok)
    c = dict(k=x, v=x, g=t(3, 5, 2, 16), beta=t(3, 5, 2), state=t(3, 2, 16, 16), path=t(3, 5, dtype=I32),
             accept=t(3, dtype=I32))
    for name, bad, err, msg in (
            ("path", t(3, 4, dtype=I32), ValueError, "path: expected shape"), ("path", None, ValueError, "required"),
            ("accept", t(3), TypeError, "accept: expected torch.int32"), ("accept", None, ValueError, "required"),
            ("state", t(3, 2, 16, 8), ValueError, "state: expected shape")):
        with pytest.raises(err, match=msg):
            kda.commit_path(**{**c, name: bad})
    with pytest.raises(ValueError, match="contiguous device tensors"):
        kda.commit_path(**c)


def test_binding_checks_verify():
    ok = dict(target=t(2, 3, 10), draft=t(2, 3, 10), tokens=t(2, 3, dtype=I32), uniforms=t(2, 3))
    for name, bad, err, msg in (
            ("target", t(2, 3, 10, dtype=torch.float16), TypeError, "bfloat16 or float32"),
            ("draft", t(2, 3, 10, dtype=BF16), TypeError, "draft: expected"), ("draft", t(2, 3, 9), ValueError, "draft: expected"),
            ("tokens", t(2, 3, dtype=torch.int64), TypeError, "tokens: expected"), ("uniforms", t(2, 2), ValueError, "uniforms"),
            ("uniforms", None, ValueError, "required"), ("parents", t(3, dtype=I32), ValueError, "parents: expected"),
            ("workspace", t(64), TypeError, "workspace: expected")):
        with pytest.raises(err, match=msg):
            kda.verify_drafts(**{**ok, name: bad})
    with pytest.raises(ValueError, match="contiguous device tensors"):
        kda.verify_drafts(**ok)
    with pytest.raises(kda.KdaError):
        kda.verify_workspace(1, 65, 100, "cpu")


@pytest.mark.parametrize("N,T,V", [(1, 2, 2 ** 32 + 5), (2 ** 32 + 1, 2, 5), (1, 2 ** 32 + 2, 5), (1, 2, 2 ** 31)])
def test_binding_refuses_sizes_past_int32(N, T, V):
    """A vocabulary of 2^32 + 5 must not run as one of 5."""
    big = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="int32"):
        kda.verify_workspace(N, T, V, "cpu")
    with pytest.raises(ValueError, match="int32"):
        kda.verify_drafts(big(N, T, V), None, big(N, T, dtype=I32), big(N, T))


def test_step_refuses_sizes_past_int32():
    big = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device="meta")  # noqa: E731
    for N, T, H in ((1, 2 ** 32 + 5, 1), (2 ** 32 + 1, 2, 1), (1, 2, 2 ** 32 + 3)):
        x, g, b, state = big(N, T, H, 16, dtype=BF16), big(N, T, H, 16), big(N, T, H), big(N, H, 16, 16)
        with pytest.raises(ValueError, match="int32"):
            kda.decode_tree(x, x, x, g, b, state)
        with pytest.raises(ValueError, match="int32"):
            kda.commit_path(x, x, g, b, state, big(N, T, dtype=I32), big(N, dtype=I32))


def test_binding_checks_cache():
    with pytest.raises(TypeError, match="values: expected"):
        kda.make_state_cache(2, 2, 16, "cpu", dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales: expected shape"):
        kda.StateCache(t(2, 2, 16, 16, dtype=torch.int8), t(2, 2, 4, dtype=torch.uint8))
    with pytest.raises(ValueError, match="values: expected shape"):
        kda.StateCache(t(2, 2, 16, 8, dtype=torch.int8), t(2, 2, 8, dtype=torch.uint8))
    c = kda.make_state_cache(2, 2, 16, "cpu")
    with pytest.raises(ValueError, match="states: expected shape"):
        kda.state_store(t(2, 3, 16, 16), c)
    with pytest.raises(TypeError, match="slots: expected"):
        kda.state_store(t(2, 2, 16, 16), c, slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous device tensors"):
        kda.state_load(c)


def test_c_abi_refusals_under_asan_and_ubsan():
    from gated_delta_rule_109_amd import build
    if not os.path.exists(build.HIPCC):
        pytest.skip("needs hipcc")
    lib = build.build_host_sanitized()
    env = dict(os.environ, LD_PRELOAD=build.san_runtime(), KDA_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:abort_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not asan",
                        "tests/test_speculative_abi.py"], env=env, cwd=ROOT, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])


def test_profiles_name_the_verification_kernels():
    assert profiling.kernel_key("void kda::(anonymous namespace)::whole_kernel<float, true>(float const*, int)") == \
        "kda::whole_kernel<float, true>"
